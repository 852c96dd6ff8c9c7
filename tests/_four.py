"""Rotated positions and keys and values in 4 bits, as plain 64-bit models (test infrastructure)."""
from __future__ import annotations

import math

import torch

from tests._paged import D, DI, Model, pool_mean, split_hi_lo

POOL = 576
# every scale a writer may give, ascending (place = its bits), and the codes' magnitudes
SCALES = torch.tensor([(m / 8 * 2.0 ** -14 if e == 0 else (1 + m / 8) * 2.0 ** (e - 15))
                       for e in range(32) for m in range(8)][:0xE3], dtype=torch.float64)
SIZES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def table(positions, dims, seed=0, base=100.0):
    """A cos_sin table [positions, dims] fp32."""
    f = base ** (-torch.arange(dims // 2, dtype=torch.float64) * 2 / dims)
    x = torch.arange(positions, dtype=torch.float64)[:, None] * f + seed
    return torch.cat([x.cos(), x.sin()], 1).float()


def pairs(dims, inter):
    """The two members of each pair."""
    j = torch.arange(dims // 2)
    return (2 * j, 2 * j + 1) if inter else (j, j + dims // 2)


def turn(x, cs, inter, inverse=False):
    """x [..., heads, d] turned in 64 bits by cs [..., dims]; also the sum of the magnitudes of what is added up."""
    dims = cs.shape[-1]
    a, b = pairs(dims, inter)
    c, s = cs[..., None, :dims // 2].double(), cs[..., None, dims // 2:].double()
    if inverse:
        s = -s
    y, mag = x.double().clone(), x.double().abs()
    p, q = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = p * c - q * s, q * c + p * s
    mag[..., a], mag[..., b] = (p * c).abs() + (q * s).abs(), (q * c).abs() + (p * s).abs()
    return y, mag


def turn_bound(y, mag):
    """Of the heads: a product and a sum rounded to fp32 (2^-24 of what is added up, and of the sum), the sum to bf16 (2^-8
    of it, or half of the smallest subnormal step)."""
    e = 2.0 ** -24 * (mag + y.abs())
    return e + 2.0 ** -8 * (y.abs() + e) + 2.0 ** -134


def turned_key(x, cs, inter):
    """A key as the cache takes it: the exact sum rounded to fp32, and that to bf16."""
    return turn(x[..., None, :], cs, inter)[0][..., 0, :].float().to(torch.bfloat16)


def nearest(v, of):
    """Places in `of` (ascending) of the numbers nearest to v, the even place of two; the last one for all beyond it."""
    v = v.clamp(max=of[-1])  # (else the distances of a huge number to the last two round to the same)
    hi = torch.searchsorted(of, v.contiguous()).clamp(max=len(of) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = (of[hi] - v).abs(), (v - of[lo]).abs()
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x):
    """x [n, 128] bf16: codes [n, 128] and scales' bits [n, 8] (integers); the nearest of all that there are."""
    y = 16 * x.double().view(-1, 8, 16)
    odd = ~torch.isfinite(y).all(2)
    y = torch.where(odd[..., None], 0.0, y)
    bits = nearest(y.abs().amax(2) / 6, SCALES)
    s = SCALES[bits][..., None]
    code = nearest(torch.where(s > 0, y.abs() / s, 0.0), SIZES)
    # (a sign bit beside a zero code stands for a zero, too)
    code = code + 8 * ((torch.signbit(y)) & (s > 0))
    return code.view(-1, 128), torch.where(odd, 0xFF, bits)


def stands_for(code, bits):
    """The values [n, 128] (64 bits) of codes and scales' bits."""
    every = torch.full((256,), math.nan, dtype=torch.float64)
    every[:len(SCALES)] = SCALES
    size = SIZES[code % 8] * torch.where(code >= 8, -1.0, 1.0)
    return (size.view(-1, 8, 16) * every[bits][..., None] / 16).view(-1, 128)


def places(t):
    """Of token t of a pool: the bytes [64] of its key's codes, of its value's, and the bytes [8] of its scales."""
    dim, g = torch.arange(0, 128, 2), torch.arange(8)
    return (t * 64 + dim // 2, 256 + dim // 16 * 32 + t * 8 + dim % 16 // 2,
            512 + g // 2 * 8 + t % 2 * 4 + t // 2 * 2 + g % 2, 544 + g * 4 + t)


def write(pool, t, k, v):
    """Token t's bytes of pool [576] (uint8): k and v (codes [128], bits [8])."""
    kc, vc, ks, vs = places(t)
    for (code, bits), c, s in ((k, kc, ks), (v, vc, vs)):
        pool[c] = (code[0::2] | code[1::2] << 4).to(torch.uint8)
        pool[s] = bits.to(torch.uint8)


def read(pool):
    """(k, v) [4, 128] in 64 bits."""
    out = []
    for half in range(2):
        rows = []
        for t in range(4):
            c, s = places(t)[half], places(t)[2 + half]
            byte = pool[c].long()
            rows.append(stands_for(torch.stack([byte % 16, byte // 16], 1).view(1, -1), pool[s].long()[None])[0])
        out.append(torch.stack(rows))
    return out


class Turned:
    """The ropes of a layer: tables of keys and of indexer keys (dims 0: none)."""

    def __init__(self, dims, dims_idx, inter, positions, apart=0):
        self.inter, self.apart = inter, apart
        self.k = table(positions, dims) if dims else None
        self.idx = table(positions, dims_idx, seed=0.5) if dims_idx else None

    def key(self, x, i):
        return x if self.k is None else turned_key(x, self.k[i], self.inter)

    def key_idx(self, x, i):
        return x if self.idx is None else turned_key(x, self.idx[i], self.inter)

    def to_gpu(self, dsa, dev="cuda"):
        def put(t):
            if t is None:
                return None
            wide = torch.full((t.shape[0], t.shape[1] + self.apart), math.nan, device=dev)
            wide[:, :t.shape[1]] = t.to(dev)
            return dsa.Rope(wide[:, :t.shape[1]], interleaved=self.inter)
        return put(self.k), put(self.idx)


class TurnedModel(Model):
    """A bf16 cache whose keys are turned on the way in."""

    def append_turned(self, ropes, k, v, k_idx):
        kt, it = k.clone(), k_idx.clone()
        for r, _, i in self.rows():
            kt[r], it[r] = ropes.key(k[r], i), ropes.key_idx(k_idx[r], i)
        self.append(kt, v, it)
        return kt, it


class Model4(TurnedModel):
    """A cache in 4 bits: kv holds the bytes, k and v the bf16 numbers that they stand for."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        k, v = quantise(self.k.view(-1, D)), quantise(self.v.view(-1, D))
        self.kv = torch.zeros(self.pages, self.page // 4, POOL, dtype=torch.uint8)
        flat = self.kv.view(-1, POOL)
        for t in range(4):
            for (code, bits), c, s in zip((k, v), places(t)[:2], places(t)[2:]):
                code = code.view(-1, 4, 128)[:, t]
                flat[:, c] = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
                flat[:, s] = bits.view(-1, 4, 8)[:, t].to(torch.uint8)
        self.k = stands_for(*k).to(torch.bfloat16).view_as(self.k)
        self.v = stands_for(*v).to(torch.bfloat16).view_as(self.v)

    def append4(self, k, v, k_idx, ropes=None):
        kt, it = (k, k_idx) if ropes is None else (k.clone(), k_idx.clone())
        for r, _, i in self.rows():
            if ropes is not None:
                kt[r], it[r] = ropes.key(k[r], i), ropes.key_idx(k_idx[r], i)
        qk, qv = quantise(kt), quantise(v)
        self.append(stands_for(*qk).to(torch.bfloat16), stands_for(*qv).to(torch.bfloat16), it)
        for r, b, i in self.rows():
            s = self.slot(b, i)
            write(self.kv.view(-1, POOL)[s // 4], s % 4, (qk[0][r], qk[1][r]), (qv[0][r], qv[1][r]))

    def to_gpu4(self, dsa, dev="cuda"):
        def put(t):
            n = t.shape[1] * t.shape[2]
            apart = self.apart * (2 if t.dtype == torch.uint8 else 1)
            flat = torch.empty(self.pages, n + apart, dtype=t.dtype, device=dev)
            view = flat.as_strided(t.shape, (n + apart, t.shape[2], 1))
            view.copy_(t)
            return view
        cache = dsa.PagedCache4(put(self.kv), put(self.k_idx), put(self.khat))
        batch = dsa.PagedBatch(self.table.to(dev), torch.tensor(self.lens, dtype=torch.int32, device=dev),
                               torch.tensor(self.cu, dtype=torch.int32, device=dev))
        return cache, batch

    def abs_values(self, pool_idx):
        """sum |v_j| over what each row attends to, and its number of keys."""
        v = self.v.view(-1, D).double().abs()
        out, n = torch.zeros(self.T, D, dtype=torch.float64), torch.zeros(self.T, dtype=torch.float64)
        for r, b, i in self.rows():
            toks = [4 * p + t for p in pool_idx[r].tolist() if p >= 0 for t in range(4)]
            toks += list(range(i // 4 * 4, i + 1))
            out[r] = v[torch.tensor([self.slot(b, t) for t in toks])].sum(0)
            n[r] = len(toks)
        return out, n


def attention4_bounds(o, av, lse, mag, sum_v, keys):
    """What the arithmetic may be off by.  Keys, values and scaled queries are exact in fp16 (a query's element under 2^-27
    of its head's largest is off by 2^-38 of that: 128 of them, 2^-31 of the largest product).  A logit is a sum of 128
    exact products in fp32 (twice 2^-24 of their magnitude each, for truncating accumulators), a weight off by that and
    2^-21 of the exponential.  P is rounded to fp16: 2^-12 of it, or 2^-25 where it is subnormal; the running maximum's
    weight is at least 1, so the normaliser is, too.  Sums of n terms in fp32 are off by n 2^-24 of their magnitude,
    twice.  o is rounded once more (2^-8 of it)."""
    ds = (2 * 128 * 2.0 ** -24 + 2.0 ** -31) * mag
    n = keys[:, None] * 2.0 ** -23
    rel = 2 * ds + 2.0 ** -20 + n + 2.0 ** -12
    off = rel[..., None] * av + 2.0 ** -25 * sum_v[:, None] + 1e-30
    return off + 2.0 ** -8 * (o.abs() + off), ds + 2.0 ** -20 + n + 2.0 ** -22 * lse.abs()


__all__ = ["D", "DI", "POOL", "SCALES", "SIZES", "Model4", "Turned", "TurnedModel", "attention4_bounds", "nearest",
           "pairs", "places", "pool_mean", "quantise", "read", "split_hi_lo", "stands_for", "table", "turn",
           "turn_bound", "turned_key", "write"]
