"""A plain model of the paged cache and of the layer over it, in Python and 64-bit CPU arithmetic (test infrastructure)."""
from __future__ import annotations

import math

import numpy as np
import torch

D, DI, HQ = 128, 64, 16


class Model:
    """Sequences of a paged cache: host copies of everything a call reads."""

    def __init__(self, new, old, page, seed, spare=3, width_extra=2, ints=False, pages_apart=0, cache_pages=None):
        """new[b] tokens appended to old[b] ones; ints: small integers (exact sums); pages_apart: extra elements
        (a multiple of 8) between pages."""
        g = torch.Generator().manual_seed(seed)
        self.new, self.old, self.page = list(new), list(old), page
        self.lens = [a + b for a, b in zip(new, old)]
        B = len(self.new)
        need = [-(-n // page) for n in self.lens]
        self.pages = cache_pages or sum(need) + spare
        self.width = max(max(need), 1) + width_extra
        perm = torch.randperm(self.pages, generator=g)
        self.table = torch.full((B, self.width), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = perm[at:at + need[b]].int()
            at += need[b]
        self.cu = [0]
        for n in self.new:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1]

        def fill(*shape):
            if ints:
                return torch.randint(-3, 4, shape, generator=g).to(torch.bfloat16)
            return torch.randn(*shape, generator=g).to(torch.bfloat16)

        self.apart = pages_apart
        self.k, self.v = fill(self.pages, page, D), fill(self.pages, page, D)
        self.k_idx = fill(self.pages, page, DI)
        self.khat = split_hi_lo(pool_mean(self.k_idx.view(-1, 4, DI))).view(self.pages, page // 4, 2 * DI)
        self.g = g
        self.fill = fill

    def slot(self, b, i):
        return int(self.table[b, i // self.page]) * self.page + i % self.page

    def rows(self):
        for b in range(len(self.new)):
            for j in range(self.new[b]):
                yield self.cu[b] + j, b, self.old[b] + j

    def to_gpu(self, dsa, dev="cuda"):
        def put(t):
            n = t.shape[1] * t.shape[2]
            flat = torch.empty(self.pages, n + self.apart, dtype=t.dtype, device=dev)
            view = flat[:, :n].view(self.pages, t.shape[1], t.shape[2]) if self.apart == 0 else \
                flat.as_strided(t.shape, (n + self.apart, t.shape[2], 1))
            view.copy_(t)
            return view
        cache = dsa.PagedCache(put(self.k), put(self.v), put(self.k_idx), put(self.khat))
        batch = dsa.PagedBatch(self.table.to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev),
                               torch.tensor(self.cu, dtype=torch.int32, device=dev))
        return cache, batch

    def append(self, k, v, k_idx):
        """The appended cache, host side (bit-exact)."""
        for r, b, i in self.rows():
            s = self.slot(b, i)
            self.k.view(-1, D)[s] = k[r]
            self.v.view(-1, D)[s] = v[r]
            self.k_idx.view(-1, DI)[s] = k_idx[r]
        for r, b, i in self.rows():
            if i % 4 == 3:
                s = self.slot(b, i)
                self.khat.view(-1, 2 * DI)[s // 4] = split_hi_lo(
                    pool_mean(self.k_idx.view(-1, DI)[s - 3:s + 1][None]))[0]

    def scores(self, q_idx, w):
        """64-bit scores of every row (one tensor per row, over its eligible pools), and the sums of magnitudes that
        bound their rounding."""
        kh = self.khat.view(-1, 2 * DI).double()
        kh = kh[:, :DI] + kh[:, DI:]
        out, mag = [], []
        for r, b, i in self.rows():
            n = i // 4
            at = torch.tensor([self.slot(b, 4 * p) // 4 for p in range(n)], dtype=torch.long)
            x = q_idx[r].double() @ kh[at].T  # [Hi, n]
            out.append((w[r].double()[:, None] * x.clamp(min=0)).sum(0))
            mag.append((w[r].double().abs()[:, None] * (q_idx[r].double().abs() @ kh[at].abs().T)).sum(0))
        return out, mag

    def attention(self, q, pool_idx, scale):
        """o, lse in 64 bits, and sum_j p_j |v_j| (what the rounding of P is relative to), sum |q||k| of the largest."""
        k, v = self.k.view(-1, D).double(), self.v.view(-1, D).double()
        o = torch.zeros(self.T, HQ, D, dtype=torch.float64)
        av = torch.zeros_like(o)
        lse = torch.zeros(self.T, HQ, dtype=torch.float64)
        mag = torch.zeros(self.T, HQ, dtype=torch.float64)
        for r, b, i in self.rows():
            toks = [4 * p + t for p in pool_idx[r].tolist() if p >= 0 for t in range(4)]
            toks += list(range(i // 4 * 4, i + 1))
            at = torch.tensor([self.slot(b, t) for t in toks])
            x = q[r].double() @ k[at].T * scale
            lse[r] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            o[r] = p @ v[at]
            av[r] = p @ v[at].abs()
            mag[r] = (q[r].double().abs() @ k[at].abs().T * scale).amax(1)
        return o, lse, av, mag


def pool_mean(x):
    """fp32 mean of the four indexer keys of each pool, in the layer's order."""
    x = x.float()
    return ((x[:, 0] + x[:, 1]) + (x[:, 2] + x[:, 3])) * 0.25


def split_hi_lo(x):
    hi = x.to(torch.bfloat16)
    return torch.cat([hi, (x - hi.float()).to(torch.bfloat16)], dim=1)


def top_pools(score, topk):
    """The row's top-k as the layer orders it: fp32 scores, ties to the lower pool, ascending, -1 padded."""
    s = score.float().numpy()
    order = np.lexsort((np.arange(len(s)), -s))[:topk]
    out = np.full(topk, -1, np.int32)
    out[:len(order)] = np.sort(order)
    return out


def random_selection(model, topk, seed, fewer=False):
    """A valid selection [T, topk]: distinct eligible pools, ascending, -1 padded (fewer: some rows keep less)."""
    rng = np.random.default_rng(seed)
    out = np.full((model.T, topk), -1, np.int32)
    for r, _, i in model.rows():
        n = min(topk, i // 4)
        if fewer and n:
            n = int(rng.integers(0, n + 1))
        out[r, :n] = np.sort(rng.choice(i // 4, n, replace=False))
    return torch.from_numpy(out)


def attention_bounds(o, av, lse, mag):
    """What the arithmetic may be off by.  Scores: 128 fp32 additions of exact products, magnitude `mag` (scaled), so
    each logit is off by at most ds = 2 * 128 * 2^-24 * mag (twice, for truncating accumulators); its weight by a
    factor 1 + ds, the exponential by 2^-21, P's rounding to bf16 by 2^-8 of each weight (half a step), the running
    sums over up to 8196 keys by less than 2^-11 in all only where nothing cancels: fp32 sums of n terms are off by
    n 2^-24 of their magnitude.  o is rounded once more (2^-8 of it)."""
    ds = 2 * 128 * 2.0 ** -24 * mag
    rel = 2 * ds + 2.0 ** -20 + 8196 * 2.0 ** -24 * 2
    o_bound = 2.0 ** -8 * o.abs() * (1 + 2.0 ** -8) + (2.0 ** -8 + rel)[..., None] * av + 1e-30
    return o_bound, ds + 2.0 ** -20 + 8196 * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
