"""The layer over a paged cache on the GPU, against a plain model in 64-bit CPU arithmetic."""
import math
import os

import numpy as np
import pytest

from tests._paged import (D, DI, HQ, Model, attention_bounds, pool_mean, random_selection, split_hi_lo, top_pools)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_context_sparse_index_gb300 as dsa
DEV = "cuda"


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def check_cache(cache, m):
    for n in ("k", "v", "k_idx", "khat"):
        assert same_bits(getattr(cache, n).cpu(), getattr(m, n)), n


# new and old tokens of the sequences: one token, a chunk, ends inside pages and pools, an idle sequence, first tokens
LAYOUTS = {
    "one": ([1], [0]),
    "second": ([1], [1]),
    "decode": ([1, 1, 1, 1, 1], [3, 16, 15, 62, 131]),
    "idle": ([1, 0, 2, 0, 7], [30, 5, 0, 0, 9]),
    "chunks": ([37, 130, 5], [0, 61, 3]),
    "pool_ends": ([2, 3, 4, 5, 6], [2, 1, 3, 7, 14]),
}


# --------------------------------------------------------------------------- append

@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_append_bit_exact(layout, page):
    m = Model(*LAYOUTS[layout], page, seed=1)
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    dsa.dsa_cache_append(cache, batch, k.to(DEV), v.to(DEV), ki.to(DEV))
    dsa.dsa_sync_status()
    m.append(k, v, ki)
    check_cache(cache, m)


def test_append_strided_rows_and_pages_and_padding():
    """Rows out of a fused projection, pages of layers that alternate, and rows behind the last sequence."""
    m = Model([5, 40, 1], [2, 7, 100], 32, seed=2, pages_apart=72)
    cache, batch = m.to_gpu(dsa)
    assert cache.k.stride(0) == 32 * D + 72
    fused = m.fill(m.T + 9, 2 * D + DI + 16)
    gpu = fused.to(DEV)
    k, v, ki = fused[:, 8:8 + D], fused[:, 8 + D:8 + 2 * D], fused[:, 16 + 2 * D:]
    dsa.dsa_cache_append(cache, batch, gpu[:, 8:8 + D], gpu[:, 8 + D:8 + 2 * D], gpu[:, 16 + 2 * D:])
    dsa.dsa_sync_status()
    m.append(k, v, ki)
    check_cache(cache, m)


def test_append_again_after_a_rejected_draft():
    """Tokens written again at earlier positions replace the slots and the pooled keys that depend on them."""
    m = Model([7], [6], 16, seed=3)
    cache, batch = m.to_gpu(dsa)
    draft = [m.fill(7, d) for d in (D, D, DI)]
    dsa.dsa_cache_append(cache, batch, *[t.to(DEV) for t in draft])
    m.append(*draft)
    m.new, m.lens, m.cu, m.T, m.old = [3], [11], [0, 3], 3, [8]
    again = [m.fill(3, d) for d in (D, D, DI)]
    batch = dsa.PagedBatch(m.table.to(DEV), torch.tensor([11], dtype=torch.int32, device=DEV),
                           torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    dsa.dsa_cache_append(cache, batch, *[t.to(DEV) for t in again])
    dsa.dsa_sync_status()
    m.append(*again)
    check_cache(cache, m)


def test_append_of_infinities_and_nan():
    """Rows are copied whatever they hold; a pool with an infinity has hi = inf and lo = inf - inf."""
    m = Model([4], [0], 16, seed=4)
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(4, D), m.fill(4, D), m.fill(4, DI)
    k[1, 5], v[2, 7], ki[0, 3], ki[1, 9] = math.inf, math.nan, math.inf, -math.inf
    dsa.dsa_cache_append(cache, batch, k.to(DEV), v.to(DEV), ki.to(DEV))
    dsa.dsa_sync_status()
    m.append(k, v, ki)
    for n in ("k", "k_idx", "v", "khat"):
        torch.testing.assert_close(getattr(cache, n).cpu(), getattr(m, n), rtol=0, atol=0, equal_nan=True)


# --------------------------------------------------------------------------- pages

class Pages:
    """The bookkeeping as plain Python."""

    def __init__(self, lens, page, num_pages, width, seed):
        rng = np.random.default_rng(seed)
        order = rng.permutation(num_pages)
        self.page, self.width = page, width
        self.lens = list(lens)
        self.table = np.full((len(lens), width), -1, np.int32)
        self.count = np.zeros(num_pages, np.int32)
        at = 0
        for s, n in enumerate(lens):
            for x in range(-(-n // page)):
                self.table[s, x] = order[at]
                self.count[order[at]] += 1
                at += 1

    def free_pages(self):
        return [int(p) for p in np.nonzero(self.count == 0)[0]]

    def reserve(self, add):
        free, need = self.free_pages(), []
        for s, a in enumerate(add):
            need.append(-(-(self.lens[s] + a) // self.page) - -(-self.lens[s] // self.page))
        taken = sum(max(n, 0) for n in need)
        if taken > len(free):
            return len(free) - taken
        for s, a in enumerate(add):
            have = -(-self.lens[s] // self.page)
            for x in range(need[s]):
                p = free.pop(0)
                self.table[s, have + x] = p
                self.count[p] = 1
            for x in range(have + min(need[s], 0), have):
                self.count[self.table[s, x]] -= 1
                self.table[s, x] = -1
            self.lens[s] += a
        return taken

    def fork(self, src, dst):
        """(pages taken, [(from, to)])"""
        free = self.free_pages()
        need = sum(1 for s in src if self.lens[s] % self.page)
        if need > len(free):
            return len(free) - need, []
        moves, lens = [], list(self.lens)
        for s, d in zip(src, dst):
            full, part = lens[s] // self.page, lens[s] % self.page
            self.table[d] = -1
            for x in range(full):
                self.table[d, x] = self.table[s, x]
                self.count[self.table[s, x]] += 1
            if part:
                p = free.pop(0)
                self.table[d, full] = p
                self.count[p] = 1
                moves.append((int(self.table[s, full]), p))
            self.lens[d] = lens[s]
        return need, moves

    def free(self, seqs):
        for s in seqs:
            for x in range(-(-self.lens[s] // self.page)):
                self.count[self.table[s, x]] -= 1
                self.table[s, x] = -1
            self.lens[s] = 0

    def compact(self):
        used = int((self.count != 0).sum())
        high = [p for p in range(used, len(self.count)) if self.count[p]]
        hole = [p for p in range(used) if not self.count[p]]
        to = dict(zip(high, hole))
        for p, q in to.items():
            self.count[q], self.count[p] = self.count[p], 0
        for s in range(self.table.shape[0]):
            for x in range(self.width):
                self.table[s, x] = to.get(int(self.table[s, x]), self.table[s, x])
        return used, list(to.items())

    def to_gpu(self):
        return dsa.PageTable(torch.from_numpy(self.table.copy()).to(DEV),
                             torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                             torch.from_numpy(self.count.copy()).to(DEV))

    def check(self, t):
        assert np.array_equal(t.page_count.cpu().numpy(), self.count)
        assert t.seq_lens.tolist() == self.lens
        assert np.array_equal(t.block_table.cpu().numpy(), self.table)


def random_cache(num_pages, page, seed=5, apart=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def new(tokens, d):
        n = tokens * d
        x = torch.randn(num_pages, n + apart, generator=g, device=DEV).to(torch.bfloat16)
        return x.as_strided((num_pages, tokens, d), (n + apart, d, 1))
    return dsa.PagedCache(new(page, D), new(page, D), new(page, DI), new(page // 4, D))


def buffers(cache):
    return [getattr(cache, n) for n in ("k", "v", "k_idx", "khat")]


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("page,apart", [(16, 0), (64, 40), (256, 0), (1024, 8)])
def test_copy_pages(page, apart):
    cache = random_cache(11, page, apart=apart)
    want = [b.clone() for b in buffers(cache)]
    src, dst = [3, 3, 0, 10, 7], [1, 4, 2, 9, 7]
    dsa.dsa_cache_copy_pages(cache, i32(src), i32(dst))
    dsa.dsa_sync_status()
    for b, w in zip(buffers(cache), want):
        w[dst] = w[src]
        assert same_bits(b, w)


def test_copy_of_no_pages_does_nothing():
    cache = random_cache(2, 16)
    dsa.dsa_cache_copy_pages(cache, i32([]), i32([]))
    dsa.dsa_sync_status()


def test_copy_of_a_page_that_is_none_is_reported():
    cache = random_cache(4, 16)
    want = [b.clone() for b in buffers(cache)]
    dsa.dsa_cache_copy_pages(cache, i32([0, 4, 1]), i32([2, 1, -1]))
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_sync_status()
    assert e.value.status == dsa.DSA_ERR_INTERNAL
    dsa.dsa_clear_status()
    for b, w in zip(buffers(cache), want):
        w[2] = w[0]
        assert same_bits(b, w)


@pytest.mark.parametrize("num_pages", [40, 255, 8200, 70001])
@pytest.mark.parametrize("page", [16, 128])
def test_reserve(num_pages, page):
    p = Pages([5 * page, 0, 3, page, 2 * page - 1], page, num_pages, 12, seed=num_pages)
    t, cache = p.to_gpu(), random_cache(num_pages, 16) if page == 16 else dsa.PagedCache.empty(num_pages, page)
    for add in ([0, 0, 0, 0, 0], [1, 1, 1, 1, 1], [0, 4 * page, 2, 0, page + 1], [page, 0, 0, 0, 0]):
        got = dsa.dsa_cache_reserve(cache, t, i32(add))
        dsa.dsa_sync_status()
        assert got.item() == p.reserve(add)
        p.check(t)


def test_reserve_without_room_changes_nothing():
    p = Pages([30, 64], 16, 8, 20, seed=1)
    t, cache = p.to_gpu(), random_cache(8, 16)
    assert dsa.dsa_cache_reserve(cache, t, i32([3, 33])).item() == p.reserve([3, 33]) == -2
    p.check(t)
    # a length the table cannot hold, and one below zero
    for add in ([320, 0], [0, -65]):
        assert dsa.dsa_cache_reserve(cache, t, i32(add)).item() == -2 ** 31
        with pytest.raises(dsa.DsaError):
            dsa.dsa_sync_status()
        dsa.dsa_clear_status()
        p.check(t)


def test_reserve_gives_pages_back():
    """Rejected drafts: sequences shrink, some to a page's end, some to nothing, while others grow in the same call."""
    p = Pages([50, 33, 16, 7, 0, 80], 16, 60, 8, seed=2)
    t, cache = p.to_gpu(), random_cache(60, 16)
    for add in ([-3, -1, 20, -7, 5, -33], [-15, 0, -20, 3, -5, -47], [40, -32, 1, -3, 0, 100]):
        assert dsa.dsa_cache_reserve(cache, t, i32(add)).item() == p.reserve(add)
        dsa.dsa_sync_status()
        p.check(t)


def test_reserve_does_not_shrink_into_a_shared_page():
    p = Pages([40, 0, 0], 16, 20, 6, seed=6)
    t, cache = p.to_gpu(), random_cache(20, 16)
    dsa.dsa_cache_fork(cache, t, i32([0]), i32([1]))
    p.fork([0], [1])
    assert dsa.dsa_cache_reserve(cache, t, i32([-1, -5, 0])).item() == p.reserve([-1, -5, 0])  # inside its own pages
    dsa.dsa_sync_status()
    p.check(t)
    assert dsa.dsa_cache_reserve(cache, t, i32([0, -10, 0])).item() == -2 ** 31  # 25 tokens: inside the second, shared page
    with pytest.raises(dsa.DsaError):
        dsa.dsa_sync_status()
    dsa.dsa_clear_status()
    p.check(t)
    assert dsa.dsa_cache_reserve(cache, t, i32([-39 + 16, -35 + 32, 0])).item() == p.reserve([-39 + 16, -35 + 32, 0])
    dsa.dsa_sync_status()
    p.check(t)


def test_reserve_of_many_sequences():
    """More sequences than a block has threads."""
    lens = [(7 * s) % 40 for s in range(2500)]
    p = Pages(lens, 16, 9000, 6, seed=9)
    t, cache = p.to_gpu(), random_cache(9000, 16)
    add = [(11 * s) % 23 for s in range(2500)]
    assert dsa.dsa_cache_reserve(cache, t, i32(add)).item() == p.reserve(add)
    dsa.dsa_sync_status()
    p.check(t)


def test_reserve_of_more_pages_than_32_bits_count():
    """1024 sequences that each ask for 2^21 pages: 2^31 in one block's sum.  Nothing changes."""
    seqs, width = 1025, 1 << 21
    cache = random_cache(40, 16)
    t = dsa.PageTable.empty(cache, seqs, width)
    t.seq_lens[1024], t.block_table[1024, 0], t.page_count[7] = 16, 7, 1
    add = torch.full((seqs,), 16 * width, dtype=torch.int32, device=DEV)
    keep = [x.clone() for x in (t.seq_lens, t.page_count)]
    for last, pages in ((0, 0), (16, 1), (-5, 0)):
        add[1024] = last
        assert dsa.dsa_cache_reserve(cache, t, add).item() == 39 - (1024 * width + pages)
        dsa.dsa_sync_status()
        assert torch.equal(t.seq_lens, keep[0]) and torch.equal(t.page_count, keep[1])
    assert t.block_table[1024, 0].item() == 7
    t.block_table[1024, 0] = -1
    assert t.block_table.amax().item() == t.block_table.amin().item() == -1


def check_moves(cache, before, moves):
    for b, w in zip(buffers(cache), before):
        for s, d in moves:
            w[d] = w[s]
        assert same_bits(b, w)


@pytest.mark.parametrize("page,apart", [(16, 0), (64, 8), (1024, 0)])
@pytest.mark.parametrize("lens", [[1], [40, 16, 0, 33], [2048, 1000, 1]])
def test_fork_then_free(lens, page, apart):
    """Children of the same parent, of a parent that ends with a page, of an empty one."""
    n = len(lens)
    p = Pages(lens + [0] * (2 * n + 1), page, 300, -(-max(lens) // page) + 2, seed=3)
    cache = random_cache(300, page, apart=apart)
    t, before = p.to_gpu(), [b.clone() for b in buffers(cache)]
    src, dst = list(range(n)) + list(range(n)), list(range(n + 1, 3 * n + 1))
    got = dsa.dsa_cache_fork(cache, t, i32(src), i32(dst))
    dsa.dsa_sync_status()
    taken, moves = p.fork(src, dst)
    assert got.item() == taken
    p.check(t)
    check_moves(cache, before, moves)
    gone = [dst[0], 0, dst[-1], dst[0]]  # one of them twice
    dsa.dsa_cache_free(cache, t, i32(gone))
    dsa.dsa_sync_status()
    p.free(gone)
    p.check(t)


def test_fork_without_room_and_bad_requests_change_nothing():
    p = Pages([20, 36, 0, 0, 0], 16, 6, 5, seed=4)
    cache = random_cache(6, 16)
    t, before = p.to_gpu(), [b.clone() for b in buffers(cache)]
    assert dsa.dsa_cache_fork(cache, t, i32([0, 1]), i32([2, 3])).item() == -1  # 5 of 6 pages are used
    dsa.dsa_sync_status()
    p.check(t)
    # a child twice, a child that lives, rows that do not exist
    for src, dst in (([0, 1], [2, 2]), ([0], [1]), ([5], [2]), ([0], [5]), ([-1], [2])):
        assert dsa.dsa_cache_fork(cache, t, i32(src), i32(dst)).item() == -2 ** 31, (src, dst)
        with pytest.raises(dsa.DsaError):
            dsa.dsa_sync_status()
        dsa.dsa_clear_status()
        p.check(t)
    check_moves(cache, before, [])
    assert dsa.dsa_cache_fork(cache, t, i32([]), i32([])).item() == 0


def test_free_of_rows_that_do_not_exist_is_reported():
    p = Pages([20, 36], 16, 6, 5, seed=4)
    t, cache = p.to_gpu(), random_cache(6, 16)
    dsa.dsa_cache_free(cache, t, i32([1, 2, -1]))
    with pytest.raises(dsa.DsaError):
        dsa.dsa_sync_status()
    dsa.dsa_clear_status()
    p.free([1])
    p.check(t)


@pytest.mark.parametrize("num_pages", [1, 7, 32, 257, 8192, 9001])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.9, 1.0])
def test_compact(num_pages, fill):
    rng = np.random.default_rng(num_pages)
    lens = [16 * int(rng.integers(1, 5)) - int(rng.integers(0, 16)) for _ in range(max(1, num_pages // 2))]
    while sum(-(-n // 16) for n in lens) > num_pages * fill:
        lens.pop()
        if not lens:
            break
    p = Pages(lens + [0, 0, 0], 16, num_pages, 6, seed=num_pages)
    if fill == 1.0:  # sequences of one page fill the rest
        for q in p.free_pages():
            p.table = np.vstack([p.table, np.full((1, 6), -1, np.int32)])
            p.table[-1, 0], p.count[q] = q, 1
            p.lens.append(16)
    cache = random_cache(num_pages, 16)
    t, before = p.to_gpu(), [b.clone() for b in buffers(cache)]
    got = dsa.dsa_cache_compact(cache, t)
    dsa.dsa_sync_status()
    used, moves = p.compact()
    assert got.tolist() == [used, len(moves)]
    p.check(t)
    for b, w in zip(buffers(cache), before):
        if moves:
            src, dst = (list(x) for x in zip(*moves))
            w[dst] = w[src]
        assert same_bits(b, w)
    again = dsa.dsa_cache_compact(cache, t)  # nothing left to move
    assert again.tolist() == [used, 0]
    p.check(t)


def test_compact_shared_pages_and_large_pages():
    p = Pages([700, 300, 513, 0, 0], 256, 40, 4, seed=8)
    cache = random_cache(40, 256, apart=16)
    t = p.to_gpu()
    dsa.dsa_cache_fork(cache, t, i32([0, 2]), i32([3, 4]))
    p.fork([0, 2], [3, 4])
    dsa.dsa_cache_free(cache, t, i32([1]))
    p.free([1])
    before = [b.clone() for b in buffers(cache)]
    dsa.dsa_cache_compact(cache, t)
    dsa.dsa_sync_status()
    _, moves = p.compact()
    p.check(t)
    check_moves(cache, before, moves)


@pytest.mark.parametrize("num_pages", [16384, 16385, 70001])
@pytest.mark.parametrize("fill", [0.0, 0.05, 0.5, 0.97, 1.0])
def test_compact_of_many_pages(num_pages, fill):
    """One CTA's plan at its largest, and a cluster's: the number of used pages is a page of the first, a middle and
    the last CTA's stretch, or of none."""
    used, width = int(num_pages * fill), 1200
    lens = [16 * min(width, used - at) - 3 for at in range(0, used, width)]
    p = Pages(lens + [0], 16, num_pages, width + 1, seed=num_pages)
    cache = random_cache(num_pages, 16)
    t, before = p.to_gpu(), [b.clone() for b in buffers(cache)]
    got = dsa.dsa_cache_compact(cache, t)
    dsa.dsa_sync_status()
    n, moves = p.compact()
    assert n == used and got.tolist() == [used, len(moves)] and bool(moves) == (0 < used < num_pages)
    p.check(t)
    for b, w in zip(buffers(cache), before):
        if moves:
            src, dst = (list(x) for x in zip(*moves))
            w[dst] = w[src]
        assert same_bits(b, w)


@pytest.mark.parametrize("num_pages", [16384, 20000])
def test_fork_of_many_children(num_pages):
    """More children than a CTA has threads, planned by one CTA and by a cluster; requests that only one of its CTAs
    can see to be bad, and one that two see half of, change nothing."""
    parents, n = 90, 9000
    lens = [1 + 7 * s % 45 for s in range(parents)]  # some end with a page
    p = Pages(lens + [0] * (n + 10), 16, num_pages, 5, seed=num_pages)
    cache = random_cache(num_pages, 16)
    t, before = p.to_gpu(), [b.clone() for b in buffers(cache)]
    order = np.random.default_rng(7).permutation(n + 10) + parents
    src, dst = [j % parents for j in range(n)], order[:n].tolist()
    for j, to in ((8191, dst[2]), (8999, dst[8191]), (0, dst[1]), (5000, 3), (7000, n + 10 + parents), (2500, -1)):
        bad = dst[:j] + [to] + dst[j + 1:]
        assert dsa.dsa_cache_fork(cache, t, i32(src), i32(bad)).item() == -2 ** 31, j
        with pytest.raises(dsa.DsaError):
            dsa.dsa_sync_status()
        dsa.dsa_clear_status()
        p.check(t)
    got = dsa.dsa_cache_fork(cache, t, i32(src), i32(dst))
    dsa.dsa_sync_status()
    taken, moves = p.fork(src, dst)
    assert got.item() == taken and taken > 8000
    p.check(t)
    froms, tos = (list(x) for x in zip(*moves))
    for b, w in zip(buffers(cache), before):
        w[tos] = w[froms]
        assert same_bits(b, w)
    left = len(p.free_pages())
    more = order[n:].tolist()
    dsa.dsa_cache_free(cache, t, i32(dst[::2]))
    p.free(dst[::2])
    p.check(t)
    assert len(p.free_pages()) > left
    got = dsa.dsa_cache_fork(cache, t, i32([0] * 10), i32(more))
    dsa.dsa_sync_status()
    assert got.item() == p.fork([0] * 10, more)[0]
    p.check(t)


@pytest.mark.parametrize("layers", [2, 33])
def test_layers_move_together(layers):
    """fork, compact and copy_pages of several layers' caches (more than one launch takes): one table, every layer's
    pages alike."""
    caches = [random_cache(24, 16, seed=l, apart=8 * (l % 3)) for l in range(layers)]
    p = Pages([40, 17, 0, 0], 16, 24, 5, seed=3)
    t, before = p.to_gpu(), [[b.clone() for b in buffers(c)] for c in caches]
    got = dsa.dsa_cache_fork(caches, t, i32([0, 1]), i32([2, 3]))
    dsa.dsa_cache_free(caches, t, i32([0]))
    info = dsa.dsa_cache_compact(tuple(caches), t)
    dsa.dsa_cache_copy_pages(caches, i32([0, 1]), i32([22, 23]))
    dsa.dsa_sync_status()
    taken, moves = p.fork([0, 1], [2, 3])
    p.free([0])
    used, more = p.compact()
    assert got.item() == taken and info.tolist() == [used, len(more)]
    p.check(t)
    for c, b in zip(caches, before):
        check_moves(c, b, moves + more + [(0, 22), (1, 23)])
    for bad in ([], None, [t], 3):
        with pytest.raises(TypeError):
            dsa.dsa_cache_compact(bad, t)


# --------------------------------------------------------------------------- indexer + top-k

def index_inputs(m, Hi, ints=True, seed=7, pad=0):
    g = torch.Generator().manual_seed(seed)
    if ints:
        q = torch.randint(-3, 4, (m.T + pad, Hi, DI), generator=g).to(torch.bfloat16)
        w = torch.randint(-1, 4, (m.T + pad, Hi), generator=g).float()
    else:
        q = torch.randn(m.T + pad, Hi, DI, generator=g).to(torch.bfloat16)
        w = torch.randn(m.T + pad, Hi, generator=g)
    return q, w


def check_topk(m, q, w, topk, got):
    scores, _ = m.scores(q, w)
    got = got.cpu().numpy()
    for r, b, i in m.rows():
        want = top_pools(scores[r], topk)
        assert np.array_equal(got[r], want), (r, b, i, got[r], want)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("Hi,topk", [(1, 1), (3, 5), (16, 8), (17, 30), (32, 512), (64, 3)])
def test_index_small_bit_exact(layout, page, Hi, topk):
    """Integer inputs: every sum is exact, ties are many, and the selection is one and the same."""
    m = Model(*LAYOUTS[layout], page, seed=11, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, Hi)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    check_topk(m, q, w, topk, got)


@pytest.mark.parametrize("new,old,page,Hi,topk", [
    ([1], [40000], 64, 8, 512), ([1, 1], [9001, 30003], 16, 32, 100), ([1] * 90, [2000 + 13 * j for j in range(90)], 64, 4, 64),
    ([3, 9, 1], [20000, 16383, 5000], 256, 16, 2048), ([130], [8191], 64, 8, 512), ([300, 20], [1000, 0], 32, 32, 77),
    ([1] * 20, [12000 + j for j in range(20)], 1024, 8, 511), ([420, 3], [9000, 30000], 64, 2, 512),
    ([310], [70000], 256, 1, 40), ([2], [70000], 64, 4, 2048), ([1, 160], [66000, 40000], 64, 2, 1000)])
def test_index_long_bit_exact(new, old, page, Hi, topk):
    m = Model(new, old, page, seed=13, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, Hi)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    check_topk(m, q, w, topk, got)


TC, PAIRS, MMA = "paged_scores_tc", "paged_scores_rows", "paged_scores"


@pytest.mark.parametrize("new,kernels", [
    ([1, 1, 200, 1, 0, 1], [TC, PAIRS]),       # a chunk among single tokens
    ([31, 32, 33, 1], [TC, PAIRS]),            # on both sides of the rule (8 heads: 32)
    ([4, 6, 9, 5, 9, 6], [TC, PAIRS]),         # one of them could be long; none is
    ([40, 150], [TC, PAIRS]),                  # all of them are
    ([31], [PAIRS]), ([32], [TC]), ([2], [PAIRS]), ([1], [MMA]), ([1] * 9, [MMA]), ([5, 1, 2, 1], [PAIRS]),
    ([3, 1, 1, 0, 0], [MMA]), ([40] + [0] * 30, [MMA]), ([70] + [0] * 30, [TC, PAIRS]),
    ([100] + [1] * 60, [TC, PAIRS]), ([40] + [1] * 60, [TC, MMA])])
def test_index_takes_each_sequence_by_its_own_rows(new, kernels):
    m = Model(new, [2500 + 700 * (j % 7) for j in range(len(new))], 64, seed=15, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 8, pad=0)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 100)
    ran = [k for k, _ in dsa.last_kernel_config()["kernels"]]
    least = torch.empty(8 * (m.width * 16 + 31) // 32 * 36 * 4 + 8 * 36 * 4, dtype=torch.uint8, device=DEV)
    small = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 100, workspace=least)
    dsa.dsa_sync_status()
    assert ran == kernels + ["paged_select"]
    check_topk(m, q, w, 100, got)
    assert torch.equal(got, small)


@pytest.mark.parametrize("new,old,kernels", [
    ([200, 1], [1000, 60000], [TC, PAIRS]),  # long enough by its rows, not by its tiles
    ([200, 1], [52000, 10], [TC, PAIRS]),    # by both
    ([200], [52000], [TC, PAIRS]), ([200], [20000], [PAIRS])])
def test_index_takes_each_sequence_by_its_own_tiles(new, old, kernels):
    m = Model(new, old, 64, seed=25, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 24)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 40)
    assert [k for k, _ in dsa.last_kernel_config()["kernels"]] == kernels + ["paged_select"]
    dsa.dsa_sync_status()
    check_topk(m, q, w, 40, got)


@pytest.mark.parametrize("case", ["zeros", "two_values", "huge", "one_high", "overflow", "negative", "runs"])
def test_index_ties_and_extreme_scores(case):
    """All scores equal; nearly all equal; magnitudes near the type's end; one score far above the rest (the bins of
    equal steps then hold everything else in one); scores that overflow to infinity; only negative scores."""
    m = Model([1, 1, 2], [30000, 9000, 17001], 64, seed=17, ints=True)
    q, w = index_inputs(m, 2, seed=18)
    w = torch.ones_like(w)
    if case == "zeros":
        w.zero_()
    elif case == "two_values":
        q.zero_()
        q[:, 0, 0] = 1
        m.k_idx.fill_(0)
        m.k_idx.view(-1, 4, DI)[::5, :, 0] = 2
    elif case == "huge":
        w *= 1e30
    elif case == "one_high":
        m.k_idx.view(-1, DI)[m.slot(0, 12345 // 4 * 4)] *= 2 ** 40
        q[:, 0, :] = 1
    elif case == "overflow":
        w *= 3e37
    elif case == "runs":  # whole pages alike: neighbours reach the threshold together, and tie
        m.k_idx.copy_(m.k_idx[:, :1].expand(-1, m.page, -1))
    else:
        w *= -1
    m.khat = split_hi_lo(pool_mean(m.k_idx.view(-1, 4, DI))).view(m.khat.shape)
    cache, batch = m.to_gpu(dsa)
    for topk in (1, 64, 700):
        got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
        dsa.dsa_sync_status()
        if case in ("zeros", "two_values", "overflow", "negative", "runs"):
            check_topk(m, q, w, topk, got)
        else:
            check_selected(m, q, w, topk, got)


def check_selected(m, q, w, topk, got):
    """Each row is a valid selection, and nothing left out scores more than a kept pool does beyond what the rounding
    of both allows.  A score's rounding: the pair holds Khat to 2^-18 of it at most (already in the 64-bit scores'
    operands here, so nothing), 128 products summed in fp32 (2 * 128 * 2^-24, twice for truncating accumulators), Hi
    more additions."""
    scores, mag = m.scores(q, w)
    got = got.cpu().numpy()
    for r, b, i in m.rows():
        n, row = i // 4, got[r]
        k = min(topk, n)
        assert np.all(row[k:] == -1) and np.all(np.diff(row[:k]) > 0) and (k == 0 or (row[0] >= 0 and row[k - 1] < n))
        if k == 0 or k == n:
            continue
        slack = (2 * 128 + q.shape[1] + 1) * 2.0 ** -24 * mag[r]
        s = scores[r]
        kept = torch.zeros(n, dtype=torch.bool)
        kept[row[:k].astype(np.int64)] = True
        assert ((s + slack)[kept].min() >= (s - slack)[~kept].max()), (r, b, i)


@pytest.mark.parametrize("Hi", [1, 2, 3, 4, 5, 7, 8, 12, 15, 16, 17, 20, 24, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("new,old,page", [([2, 7, 11], [1200, 37, 517], 32), ([21, 3], [2047, 5000], 256),
                                          ([23], [1500], 1024)])
def test_index_of_every_number_of_heads(Hi, new, old, page):
    """Groups of 256 / Hi rows whose heads lie across the columns in every alignment."""
    m = Model(new, old, page, seed=14, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, Hi)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 33)
    assert any(k == PAIRS for k, _ in dsa.last_kernel_config()["kernels"])
    dsa.dsa_sync_status()
    check_topk(m, q, w, 33, got)


@pytest.mark.parametrize("page", [16, 128, 1024])
@pytest.mark.parametrize("new,old", [([1, 2, 1], [3000, 701, 40]), ([1, 2, 5], [3000, 701, 40]),
                                     ([130, 1, 27], [3001, 5000, 0])])
def test_index_reads_nothing_it_may_not_see(new, old, page):
    """NaN and infinities in every pooled key that no row may see: pools past a row's end, later pages, other pages."""
    m = Model(new, old, page, seed=16, ints=True)
    seen = torch.zeros(m.khat.shape[0] * m.khat.shape[1], dtype=torch.bool)
    for b, n in enumerate(m.lens):
        for p in range((n - 1) // 4):
            seen[m.slot(b, 4 * p) // 4] = True
    flat = m.khat.view(-1, 2 * DI)
    flat[~seen] = math.nan
    flat[(~seen).nonzero()[::2, 0], :DI] = math.inf
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 8)
    for topk in (5, 600):
        got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
        dsa.dsa_sync_status()
        check_topk(m, q, w, topk, got)


@pytest.mark.parametrize("new", [[1, 1, 1], [8], [40]])
@pytest.mark.parametrize("topk", [7, 512])
def test_index_of_a_row_of_nan_stays_in_bounds(new, topk):
    """A row whose weights are NaN selects topk different pools that it may see, ascending; the rows beside it are as ever."""
    m = Model(new, [9000 + 4 * j for j in range(len(new))], 64, seed=20, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 4)
    bad = w.clone()
    bad[1] = math.nan
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), bad.to(DEV), topk).cpu()
    dsa.dsa_sync_status()
    (_, _, i), = [x for x in m.rows() if x[0] == 1]
    row = got[1].long()
    assert row[0] >= 0 and row[-1] < i // 4 and torch.all(row[1:] > row[:-1])
    good = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk).cpu()
    got[1] = good[1]
    assert torch.equal(got, good)


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("old,page,topk", [(600, 16, 64), (0, 64, 200), (1000, 32, 512)])
def test_index_of_many_short_rows(ints, old, page, topk):
    """More rows than the chip takes at once, in a table that is never wider than 8 * topk pools."""
    m = Model([900], [old], page, seed=26, ints=ints)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 4, ints=ints)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    (check_topk if ints else check_selected)(m, q, w, topk, got)


@pytest.mark.parametrize("case", ["zeros", "two_values", "one_high", "negative", "few_values"])
@pytest.mark.parametrize("topk", [1, 300, 512])
def test_index_ties_of_many_rows(case, topk):
    """Rows by the hundred go a warp each; rows whose list of candidates cannot hold the ties, or comes out too short,
    are left to the other kernel."""
    m = Model([330], [12001], 64, seed=18, ints=True)
    q, w = index_inputs(m, 1, seed=19)
    w = torch.ones_like(w)
    ki = m.k_idx.view(-1, 4, DI)
    if case == "zeros":
        w[::2] = 0  # every other row
    elif case == "two_values":
        q.zero_()
        q[:, 0, 0] = 1
        m.k_idx.fill_(0)
        ki[::3, :, 0] = 2
    elif case == "one_high":
        ki[m.slot(0, 4000) // 4] *= 2 ** 20
    elif case == "negative":
        w *= -1
    else:
        q[:, :, 4:] = 0  # scores of few values: the k-th ties with hundreds
    m.khat = split_hi_lo(pool_mean(ki)).view(m.khat.shape)
    cache, batch = m.to_gpu(dsa)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    check_topk(m, q, w, topk, got)


@pytest.mark.parametrize("topk", [512, 2000])
def test_index_of_rows_longer_than_a_segment(topk):
    """Past 2^17 pools the kept bits are written a segment at a time, carrying the ties: one row by its list, one (all
    scores equal) from the row itself, one whose ties begin in the second segment."""
    m = Model([1, 1, 1], [600000, 560001, 540003], 1024, seed=20, ints=True)
    q, w = index_inputs(m, 1, seed=21)
    w[0], w[1], w[2] = 1, 0, 1
    q[2] = 0
    q[2, 0, 0] = 1
    page = m.table[2].tolist()
    for x in range(525 if topk == 512 else 520, 527):  # the last sequence's high scores: pools past 2^17, all equal
        m.k_idx[page[x]] = 0
        m.k_idx[page[x], :, 0] = 8
    m.khat = split_hi_lo(pool_mean(m.k_idx.view(-1, 4, DI))).view(m.khat.shape)
    cache, batch = m.to_gpu(dsa)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    check_topk(m, q, w, topk, got)


@pytest.mark.parametrize("Hi", [64, 2])
def test_index_of_eight_rows_past_2_28_pools(Hi):
    """A table of 2^20 + 1 pages of 1024 tokens, all but the last one page of zeros: the passes' least, eight rows, then
    has more tiles than a pass of 2^31 scores, and the best pools lie in its last tiles."""
    page, width, topk, rows = 1024, (1 << 20) + 1, 8, 8
    cache = dsa.PagedCache.empty(2, page)
    cache.khat.zero_()
    best = torch.randperm(256, generator=torch.Generator().manual_seed(4)).float()
    cache.khat[1, :, 0] = best.to(torch.bfloat16).to(DEV)
    table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    n = width * page
    batch = dsa.PagedBatch(table, i32([n]), i32([0, rows]))
    q = torch.zeros(rows, Hi, DI, dtype=torch.bfloat16, device=DEV)
    q[:, 0, 0] = 1
    ws = torch.full((dsa.paged_index_topk_workspace_size(rows, width, page),), 255, dtype=torch.uint8, device=DEV)
    got = dsa.dsa_paged_index_topk(cache, batch, q, torch.ones(rows, Hi, device=DEV), topk, workspace=ws)
    dsa.dsa_sync_status()
    assert [k for k, _ in dsa.last_kernel_config()["kernels"]] == [PAIRS, "paged_select"]
    for r in range(rows):
        first = (width - 1) * page // 4
        mine = best[:(n - rows + r) // 4 - first]
        want = sorted(first + j for j in mine.topk(topk).indices.tolist())
        assert got[r].tolist() == want, r


@pytest.mark.parametrize("Hi,topk", [(32, 512), (5, 100)])
@pytest.mark.parametrize("new,old", [([1, 1, 1], [33000, 4097, 12003]), ([140], [10000]), ([350], [10000])])
def test_index_real_values(new, old, Hi, topk):
    m = Model(new, old, 64, seed=19)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, Hi, ints=False)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    again = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), topk)
    dsa.dsa_sync_status()
    assert torch.equal(got, again)
    check_selected(m, q, w, topk, got)


def test_index_does_not_depend_on_the_workspace_and_leaves_padding():
    """The least workspace (8 rows at a time) and the recommended one; rows behind the last sequence stay."""
    m = Model([30, 1, 8], [3000, 777, 5000], 64, seed=23, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 8, pad=6)
    q, w = q.to(DEV), w.to(DEV)
    out = torch.full((m.T + 6, 50), 77, dtype=torch.int32, device=DEV)
    full = dsa.dsa_paged_index_topk(cache, batch, q, w, 50, pool_idx=out.clone())
    least = torch.empty(8 * (m.width * 16 + 31) // 32 * 36 * 4 + 8 * 36 * 4, dtype=torch.uint8, device=DEV)
    small = dsa.dsa_paged_index_topk(cache, batch, q, w, 50, pool_idx=out.clone(), workspace=least)
    dsa.dsa_sync_status()
    assert torch.equal(full, small)
    assert torch.all(full[m.T:] == 77)
    check_topk(m, q.cpu(), w.cpu(), 50, full)


def test_index_equals_the_contiguous_call():
    """A whole prompt as one chunk: the same pools as dsa_index_topk."""
    m = Model([3001], [0], 64, seed=29, ints=True)
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    dsa.dsa_cache_append(cache, batch, k.to(DEV), v.to(DEV), ki.to(DEV))
    q, w = index_inputs(m, 8)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 64)
    want = dsa.dsa_index_topk(q.to(DEV), ki.to(DEV), w.to(DEV), chunk=256, topk=64)
    dsa.dsa_sync_status()
    assert torch.equal(got, want)


# --------------------------------------------------------------------------- attention

def check_attention(m, q, sel, scale, o, lse):
    ro, rl, av, mag = m.attention(q, sel, scale)
    bo, bl = attention_bounds(ro, av, rl, mag)
    T = m.T
    err = (o[:T].cpu().double() - ro).abs()
    assert torch.all(err <= bo), (err / bo).max()
    err = (lse[:T].cpu().double() - rl).abs()
    assert torch.all(err <= bl), (err / bl).max()


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("topk", [1, 15, 16, 64])
def test_attention_small(layout, page, topk):
    m = Model(*LAYOUTS[layout], page, seed=31)
    cache, batch = m.to_gpu(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, topk, seed=1)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    check_attention(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("rows", [1, 2, 14, 16, 25, 38, 39, 60, 76, 100, 128, 152, 153, 228, 229, 400])
@pytest.mark.parametrize("topk", [512, 300, 96, 80])
def test_attention_every_split(rows, topk):
    """Every number of CTAs per row; rows that keep fewer pools than the others leave CTAs without keys."""
    m = Model([1] * rows, [50 + 37 * j % 3000 for j in range(rows)], 64, seed=37)
    cache, batch = m.to_gpu(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, topk, seed=rows, fewer=True)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    o2, lse2 = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    assert same_bits(o, o2) and torch.equal(lse, lse2)
    check_attention(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("new,old,topk", [([1], [9000], 2048), ([3], [70000], 1000), ([200], [8200], 2048),
                                          ([19], [8300], 2048), ([60], [9000], 1500)])
def test_attention_long(new, old, topk):
    m = Model(new, old, 128, seed=41, pages_apart=24)
    cache, batch = m.to_gpu(dsa)
    q, sel = m.fill(m.T, HQ, D) * 2, random_selection(m, topk, seed=2)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), scale=0.1)
    dsa.dsa_sync_status()
    check_attention(m, q, sel, 0.1, o, lse)


@pytest.mark.parametrize("rows", [3, 100, 500])
def test_attention_reads_nothing_it_does_not_attend_to(rows):
    """NaN and infinities in every slot that no row attends to, positions behind the last token among them."""
    m = Model([1] * rows, [40 + 3 * j for j in range(rows)], 16, seed=43)
    sel = random_selection(m, 8, seed=3)
    seen = torch.zeros(m.pages * m.page, dtype=torch.bool)
    for r, b, i in m.rows():
        for t in [4 * p + e for p in sel[r].tolist() if p >= 0 for e in range(4)] + list(range(i // 4 * 4, i + 1)):
            seen[m.slot(b, t)] = True
    m.k.view(-1, D)[~seen] = math.nan
    m.v.view(-1, D)[~seen] = math.inf
    cache, batch = m.to_gpu(dsa)
    q = m.fill(m.T, HQ, D)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    check_attention(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("rows", [2, 200])
def test_attention_leaves_padding_and_given_outputs(rows):
    m = Model([1] * rows, [100] * rows, 32, seed=47)
    cache, batch = m.to_gpu(dsa)
    q = m.fill(m.T + 5, HQ, D)
    sel = torch.cat([random_selection(m, 16, seed=4), torch.zeros(5, 16, dtype=torch.int32)])
    o = torch.full((m.T + 5, HQ, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((m.T + 5, HQ), 5.0, device=DEV)
    dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), o=o, lse=lse)
    dsa.dsa_sync_status()
    assert torch.all(o[m.T:] == 3.0) and torch.all(lse[m.T:] == 5.0)
    check_attention(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("what", ["page", "page_high", "length", "offsets", "selection", "order"])
@pytest.mark.parametrize("rows", [4, 300])
def test_what_is_out_of_range_is_reported_and_not_followed(what, rows):
    """A page number that is none, a length past the table, offsets against lengths, a pool that is not eligible: the
    status says so, the other rows are right."""
    m = Model([1] * rows, [200 + j % 50 for j in range(rows)], 16, seed=53)
    bad = 2
    sel = random_selection(m, 16, seed=5)
    q = m.fill(m.T, HQ, D)
    good = Model([1] * rows, [200 + j % 50 for j in range(rows)], 16, seed=53)
    if what == "page":
        m.table[bad, int(sel[bad, 0]) // 4] = -1
    elif what == "page_high":
        m.table[bad, int(sel[bad, 0]) // 4] = m.pages
    elif what == "length":
        m.lens[bad] = m.width * 16 + 1
    elif what == "offsets":
        m.lens[bad] = 0
    elif what == "selection":
        sel[bad, 15] = (m.lens[bad] - 1) // 4
    else:
        sel[bad, 1] = sel[bad, 0]
    cache, batch = m.to_gpu(dsa)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_sync_status()
    assert e.value.status == dsa.DSA_ERR_INTERNAL
    dsa.dsa_clear_status()
    ok = [r for r in range(rows) if r != bad]
    sel[bad] = -1
    ro, rl, av, mag = good.attention(q, sel, 1 / math.sqrt(D))
    bo, bl = attention_bounds(ro, av, rl, mag)
    assert torch.all((o.cpu().double() - ro).abs()[ok] <= bo[ok])
    assert torch.all((lse.cpu().double() - rl).abs()[ok] <= bl[ok])
    if what in ("page", "page_high", "length", "offsets"):  # the indexer and the append follow the same numbers
        qi, w = index_inputs(m, 4)
        if what in ("page", "page_high"):
            m.table[bad] = -1 if what == "page" else m.pages
            batch.block_table.copy_(m.table)
        dsa.dsa_paged_index_topk(cache, batch, qi.to(DEV), w.to(DEV), 16)
        with pytest.raises(dsa.DsaError):
            dsa.dsa_sync_status()
        dsa.dsa_clear_status()
        dsa.dsa_cache_append(cache, batch, *[m.fill(m.T, d).to(DEV) for d in (D, D, DI)])
        with pytest.raises(dsa.DsaError):
            dsa.dsa_sync_status()
        dsa.dsa_clear_status()


@pytest.mark.parametrize("what", ["page", "page_high", "length", "offsets", "backwards", "past_the_rows"])
@pytest.mark.parametrize("new,kernels", [([1, 1, 1, 1], [MMA]), ([5, 7, 3, 4], [PAIRS]), ([40, 50, 60, 33], [TC, PAIRS])])
def test_index_out_of_range_on_every_kernel(what, new, kernels):
    """As above for the three kernels of the scores, and offsets that run backwards or past the call's rows."""
    old = [900, 1300, 700, 1111]
    m, good = (Model(new, old, 32, seed=54, ints=True) for _ in range(2))
    q, w = index_inputs(m, 8)
    bad = 2
    if what in ("page", "page_high"):
        m.table[bad] = -1 if what == "page" else m.pages
    elif what == "length":
        m.lens[bad] = m.width * 32 + 1
    elif what == "offsets":
        m.lens[bad] = 0
    elif what == "backwards":
        m.cu[bad], m.cu[bad + 1] = m.cu[bad + 1], m.cu[bad]
    else:
        m.cu[-1] += 1 << 20
    cache, batch = m.to_gpu(dsa)
    got = torch.full((m.T, 20), -7, dtype=torch.int32, device=DEV)
    dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 20, pool_idx=got)
    assert [k for k, _ in dsa.last_kernel_config()["kernels"]] == kernels + ["paged_select"]
    got = got.cpu()
    if what != "backwards":  # (rows that another sequence then claims too may be anybody's, with or without a status)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_sync_status()
        assert e.value.status == dsa.DSA_ERR_INTERNAL
    dsa.dsa_clear_status()
    assert torch.all((got >= -7) & (got < 1400))
    scores, _ = good.scores(q, w)
    hit = {"backwards": (1, 2, 3), "past_the_rows": (3,)}.get(what, (bad,))
    for r, b, i in good.rows():
        if b not in hit:
            assert np.array_equal(got[r].numpy(), top_pools(scores[r], 20)), (r, b, i)


@pytest.mark.parametrize("cu,first_bad", [([-3, 5, 8], (0, 5)), ([-3, -3, 8], (0, 8)), ([0, 5, 9], (5, 8)),
                                          ([0, 5, 3], (8, 8)), ([0, -2, 8], (0, 8))])
def test_offsets_that_leave_the_rows(cu, first_bad):
    """Offsets below 0, past the call's rows, and backwards: the append writes nothing, the rows of such a sequence get
    no selection and no output, and the status says so; the other sequence's rows are right."""
    m, good = (Model([5, 3], [59, 41], 16, seed=55, ints=True) for _ in range(2))
    m.cu, (lo, hi) = cu, first_bad
    cache, batch = m.to_gpu(dsa)

    def reported():
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_sync_status()
        assert e.value.status == dsa.DSA_ERR_INTERNAL
        dsa.dsa_clear_status()

    new = [m.fill(m.T, d).to(DEV) for d in (D, D, DI)]
    assert new[0].shape[0] == 8
    dsa.dsa_cache_append(cache, batch, *new)
    reported()
    check_cache(cache, m)
    if cu == [0, 5, 3]:  # (rows 5..7 are then behind the last sequence)
        return
    q, w = index_inputs(m, 4)
    sel = torch.full((8, 6), -7, dtype=torch.int32, device=DEV)
    dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 6, pool_idx=sel)
    reported()
    assert torch.all(sel[lo:hi] == -1)
    qa = m.fill(m.T, HQ, D)
    o = torch.full((8, HQ, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((8, HQ), 5.0, device=DEV)
    dsa.dsa_paged_sparse_attn_fwd(cache, batch, qa.to(DEV), sel, o=o, lse=lse)
    reported()
    assert torch.all(o[lo:hi] == 3.0) and torch.all(lse[lo:hi] == 5.0)
    ok = [r for r in range(8) if not lo <= r < hi]
    scores, _ = good.scores(q, w)
    for r in ok:
        assert np.array_equal(sel[r].cpu().numpy(), top_pools(scores[r], 6)), r
    ro, rl, av, mag = good.attention(qa, sel.cpu(), 1 / math.sqrt(D))
    bo, bl = attention_bounds(ro, av, rl, mag)
    assert torch.all((o.cpu().double() - ro).abs()[ok] <= bo[ok])
    assert torch.all((lse.cpu().double() - rl).abs()[ok] <= bl[ok])


# --------------------------------------------------------------------------- together

def test_prompts_in_chunks_then_tokens_with_forks_and_compaction():
    """As a server runs it: prompts arrive in chunks, tokens follow one by one, sequences are forked and freed, the
    cache is compacted; every step's selection and attention are those of the contiguous calls on the same tokens."""
    page, topk, Hi = 16, 24, 4
    cache = random_cache(120, page)
    t = dsa.PageTable.empty(cache, max_seqs=4, max_pages=20)
    g = torch.Generator().manual_seed(3)

    def tokens(n):
        k, v = (torch.randn(n, D, generator=g).to(torch.bfloat16) for _ in range(2))
        ki = torch.randint(-3, 4, (n, DI), generator=g).to(torch.bfloat16)
        qi = torch.randint(-3, 4, (n, Hi, DI), generator=g).to(torch.bfloat16)
        w = torch.randint(0, 4, (n, Hi), generator=g).float()
        return [x.to(DEV) for x in (k, v, ki, qi, w, torch.randn(n, HQ, D, generator=g).to(torch.bfloat16))]

    hist = {s: None for s in range(4)}

    def step(adds):
        add = [adds.get(s, 0) for s in range(4)]
        assert dsa.dsa_cache_reserve(cache, t, i32(add)).item() >= 0
        cu = i32(np.concatenate([[0], np.cumsum(add)]))
        new = tokens(sum(add))
        batch = dsa.PagedBatch(t.block_table, t.seq_lens, cu)
        dsa.dsa_cache_append(cache, batch, *new[:3])
        pool_idx = dsa.dsa_paged_index_topk(cache, batch, new[3], new[4], topk)
        o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, new[5], pool_idx)
        dsa.dsa_sync_status()
        at = 0
        for s, n in enumerate(add):
            if n == 0:
                continue
            mine = [x[at:at + n] for x in new]
            hist[s] = mine if hist[s] is None else [torch.cat(p) for p in zip(hist[s], mine)]
            k, v, ki, qi, w, q = hist[s]
            S = k.shape[0]
            want = dsa.dsa_index_topk(qi, ki, w, chunk=64, topk=topk)
            assert torch.equal(pool_idx[at:at + n], want[S - n:])
            wo, wl = dsa.dsa_sparse_attn_fwd(q, k, v, want)
            torch.testing.assert_close(o[at:at + n].float(), wo[S - n:].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
            torch.testing.assert_close(lse[at:at + n], wl[S - n:], rtol=1e-5, atol=1e-5)
            at += n

    step({0: 50, 1: 3})
    step({0: 61, 1: 17})
    for _ in range(6):
        step({0: 1, 1: 1})
    dsa.dsa_cache_fork(cache, t, i32([0, 0]), i32([2, 3]))
    hist[2] = hist[3] = hist[0]
    for _ in range(9):
        step({0: 1, 1: 1, 2: 1, 3: 1})
    dsa.dsa_cache_free(cache, t, i32([0, 1]))
    hist[0] = hist[1] = None
    used, moved = dsa.dsa_cache_compact(cache, t).tolist()
    assert used == int((t.page_count != 0).sum()) and torch.all(t.page_count[:used] > 0)
    for _ in range(5):
        step({2: 1, 3: 2})
    step({0: 30, 2: 5, 3: 1})
    dsa.dsa_cache_free(cache, t, i32([0, 2, 3]))
    assert torch.all(t.page_count == 0) and torch.all(t.block_table == -1) and torch.all(t.seq_lens == 0)


def test_decoding_step_in_a_replayed_graph():
    """reserve, append, indexer and attention captured once and replayed with new tokens and growing lengths; two
    graphs share one workspace."""
    m = Model([1] * 5, [20, 333, 64, 63, 100], 16, seed=59, ints=True, spare=40, width_extra=4)
    cache, batch = m.to_gpu(dsa)
    B, Hi, topk = 5, 8, 16
    lens0 = torch.tensor(m.old, dtype=torch.int32, device=DEV)
    count = torch.zeros(m.pages, dtype=torch.int32)
    table = m.table.clone()
    for b, n in enumerate(m.old):
        table[b, -(-n // 16):] = -1
    for p in table.flatten().tolist():
        if p >= 0:
            count[p] += 1
    t = dsa.PageTable(table.to(DEV), lens0.clone(), count.to(DEV))
    cu = i32(range(B + 1))
    batch = dsa.PagedBatch(t.block_table, t.seq_lens, cu)
    k, v, ki = (torch.empty(B, d, dtype=torch.bfloat16, device=DEV) for d in (D, D, DI))
    qi = torch.empty(B, Hi, DI, dtype=torch.bfloat16, device=DEV)
    w, q = torch.empty(B, Hi, device=DEV), torch.empty(B, HQ, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(dsa.paged_index_topk_workspace_size(B, t.max_pages, 16),
                         dsa.cache_workspace_size(m.pages, B)), dtype=torch.uint8, device=DEV)
    outs = [(torch.empty(B, topk, dtype=torch.int32, device=DEV), torch.empty_like(q),
             torch.empty(B, HQ, device=DEV), i32([0])) for _ in range(2)]
    one = i32([1] * B)

    def step(out):
        dsa.dsa_cache_reserve(cache, t, one, result=out[3], workspace=ws)
        dsa.dsa_cache_append(cache, batch, k, v, ki)
        dsa.dsa_paged_index_topk(cache, batch, qi, w, topk, pool_idx=out[0], workspace=ws)
        dsa.dsa_paged_sparse_attn_fwd(cache, batch, q, out[0], o=out[1], lse=out[2])

    keep = [x.clone() for x in (t.block_table, t.seq_lens, t.page_count)]
    for x in (k, v, ki, qi, w, q):
        x.zero_()
    step(outs[0])  # warm-up
    torch.cuda.synchronize()
    for x, y in zip((t.block_table, t.seq_lens, t.page_count), keep):
        x.copy_(y)
    graphs = []
    for out in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(out)
        graphs.append(gr)
    for it in range(24):
        new = [m.fill(B, D), m.fill(B, D), m.fill(B, DI), m.fill(B, Hi, DI), m.fill(B, Hi).float().abs(), m.fill(B, HQ, D)]
        for dst, src in zip((k, v, ki, qi, w, q), new):
            dst.copy_(src)
        graphs[it % 2].replay()
        dsa.dsa_sync_status()
        m.table = t.block_table.cpu()
        m.append(*new[:3])
        out = outs[it % 2]
        check_topk(m, new[3], new[4], topk, out[0])
        check_attention(m, new[5], out[0].cpu(), 1 / math.sqrt(D), out[1], out[2])
        m.old = [n + 1 for n in m.old]
        m.lens = [n + 1 for n in m.lens]


def test_a_step_that_found_too_few_pages_overwrites_nothing():
    """reserve and append captured and replayed until the pages run out: the refused steps leave every live token (a
    forked sibling's among them) as it was, and say so; with pages free again the next replay goes on."""
    cache = random_cache(8, 16)
    t = dsa.PageTable.empty(cache, max_seqs=3, max_pages=6)
    cu = i32([0, 40, 40, 40])
    new = [torch.randn(40, d, device=DEV).to(torch.bfloat16) for d in (D, D, DI)]
    taken, add = i32([0]), i32([48, 0, 48])
    assert dsa.dsa_cache_reserve(cache, t, add).item() == 6
    dsa.dsa_cache_fork(cache, t, i32([0]), i32([1]))  # three full pages, shared
    ws = torch.empty(dsa.cache_workspace_size(8, 3), dtype=torch.uint8, device=DEV)
    cu.copy_(i32([0, 1, 2, 2]))
    add.copy_(i32([1, 1, 0]))
    batch = dsa.PagedBatch(t.block_table, t.seq_lens, cu)
    k, v, ki = (x[:2] for x in new)

    def step():
        dsa.dsa_cache_reserve(cache, t, add, result=taken, workspace=ws)
        dsa.dsa_cache_append(cache, batch, k, v, ki, reserved=taken)

    step()  # warm-up: the last two pages
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(15):
        g.replay()
    dsa.dsa_sync_status()
    assert taken.item() == 0 and t.seq_lens.tolist() == [64, 64, 48] and torch.all(t.page_count > 0)
    keep = [x.clone() for x in buffers(cache) + [t.block_table, t.seq_lens, t.page_count]]
    for add_now in ([1, 1, 0], [0, 0, 200]):  # no page left; more than a row of the table holds
        add.copy_(i32(add_now))
        cu.copy_(i32([0, 1, 2, 2] if add_now[0] else [0, 0, 0, 2]))
        g.replay()
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_sync_status()
        assert e.value.status == dsa.DSA_ERR_INTERNAL
        dsa.dsa_clear_status()
        assert taken.item() == (-2 if add_now[0] else -2 ** 31)
        for x, y in zip(buffers(cache) + [t.block_table, t.seq_lens, t.page_count], keep):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    dsa.dsa_cache_free(cache, t, i32([2]))
    add.copy_(i32([1, 1, 0]))
    cu.copy_(i32([0, 1, 2, 2]))
    g.replay()
    dsa.dsa_sync_status()
    assert taken.item() == 2 and t.seq_lens.tolist() == [65, 65, 0]
    for s_ in (0, 1):
        page = t.block_table[s_, 4].item()
        assert same_bits(cache.k[page, 0], k[s_]) and same_bits(cache.v[page, 0], v[s_])
    for bad in (i32([0, 0]), torch.zeros(1, device=DEV), taken.cpu()):
        with pytest.raises((TypeError, ValueError)):
            dsa.dsa_cache_append(cache, batch, k, v, ki, reserved=bad)


def test_page_operators_in_a_replayed_graph():
    """fork, reserve, free and compact captured once and replayed on changing tables."""
    p = Pages([40, 33, 0, 0, 0], 16, 30, 6, seed=12)
    cache = random_cache(30, 16)
    t = p.to_gpu()
    src, dst, add, gone = i32([0, 1]), i32([2, 3]), i32([0, 0, 20, 1, 0]), i32([0, 4])
    ws = torch.empty(dsa.cache_workspace_size(30, 5, 2), dtype=torch.uint8, device=DEV)
    out = [i32([0]), i32([0]), i32([0, 0])]

    def step():
        dsa.dsa_cache_fork(cache, t, src, dst, result=out[0], workspace=ws)
        dsa.dsa_cache_reserve(cache, t, add, result=out[1], workspace=ws)
        dsa.dsa_cache_free(cache, t, gone)
        dsa.dsa_cache_compact(cache, t, result=out[2], workspace=ws)

    keep = [x.clone() for x in (t.block_table, t.seq_lens, t.page_count)]
    step()  # warm-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for x, y in zip((t.block_table, t.seq_lens, t.page_count), keep):
        x.copy_(y)
    for s, d, a, f in (([0, 1], [2, 3], [0, 0, 20, 1, 0], [0, 4]), ([2, 3], [0, 4], [5, -33, 0, 0, 7], [2, 2]),
                       ([4, 0], [1, 2], [0, 0, 0, -2, 0], [3, 0])):
        for x, y in ((src, s), (dst, d), (add, a), (gone, f)):
            x.copy_(i32(y))
        before = [b.clone() for b in buffers(cache)]
        g.replay()
        dsa.dsa_sync_status()
        taken, moves = p.fork(s, d)
        assert out[0].item() == taken and out[1].item() == p.reserve(a)
        p.free(f)
        used, more = p.compact()
        assert out[2].tolist() == [used, len(more)]
        p.check(t)
        check_moves(cache, before, moves + more)


@pytest.mark.parametrize("rows", [200, 20])
def test_tcgen05_scores_time_out_and_the_next_call_is_right(rows):
    """With fault injection the tcgen05 scores' producer issues no copies: every bounded wait runs out, the call
    reports DSA_ERR_TIMEOUT, and the context stays usable."""
    m = Model([rows], [3000], 64, seed=62, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 8)
    dsa.dsa_clear_status()
    os.environ["DSA_FAULT_INJECT"] = "timeout"
    try:
        dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 64)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_sync_status()
        assert e.value.status == dsa.DSA_ERR_TIMEOUT
    finally:
        del os.environ["DSA_FAULT_INJECT"]
    dsa.dsa_clear_status()
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 64)
    dsa.dsa_sync_status()
    check_topk(m, q, w, 64, got)


def test_calls_on_a_stream_of_their_own():
    m = Model([1, 40], [5000, 100], 64, seed=61, ints=True)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 8)
    q, w, qa = q.to(DEV), w.to(DEV), m.fill(m.T, HQ, D).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pool_idx = dsa.dsa_paged_index_topk(cache, batch, q, w, 64, stream=side)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, qa, pool_idx, stream=side)
    side.synchronize()
    dsa.dsa_sync_status(side)
    check_topk(m, q.cpu(), w.cpu(), 64, pool_idx)
    check_attention(m, qa.cpu(), pool_idx.cpu(), 1 / math.sqrt(D), o, lse)


def test_large_cache_offsets_past_32_bits():
    """Pages beyond 2^32 bytes (and 2^31 elements) of a buffer are reached."""
    page, pages = 1024, 20000  # k: 5.2 GB, 2.6e9 elements
    cache = dsa.PagedCache.empty(pages, page)
    n = 3 * page + 5
    table = i32([pages - 1, 0, pages - 2, 1]).view(1, 4)
    cu = i32([0, n])
    batch = dsa.PagedBatch(table, i32([n]), cu)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(n, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    ki = torch.randint(-3, 4, (n, DI), generator=g, device=DEV).to(torch.bfloat16)
    dsa.dsa_cache_append(cache, batch, k, v, ki)
    assert same_bits(cache.k[pages - 1], k[:page]) and same_bits(cache.v[pages - 2], v[2 * page:3 * page])
    qi = torch.randint(-3, 4, (n, 4, DI), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randint(0, 4, (n, 4), generator=g, device=DEV).float()
    got = dsa.dsa_paged_index_topk(cache, batch, qi, w, 64)
    want = dsa.dsa_index_topk(qi, ki, w, chunk=256, topk=64)
    assert torch.equal(got, want)
    q = torch.randn(n, HQ, D, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, q, got)
    wo, wl = dsa.dsa_sparse_attn_fwd(q, k, v, want)
    dsa.dsa_sync_status()
    torch.testing.assert_close(o.float(), wo.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    torch.testing.assert_close(lse, wl, rtol=1e-5, atol=1e-5)
    dsa.dsa_cache_copy_pages(cache, i32([pages - 1]), i32([pages - 3]))
    dsa.dsa_sync_status()
    assert same_bits(cache.k[pages - 3], k[:page])


def test_calls_record_what_they_ran():
    m = Model([1], [100], 16, seed=67)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 4)
    dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 8)
    c = dsa.last_kernel_config()
    assert c["entry"] == "dsa_paged_index_topk" and [k for k, _ in c["kernels"]] == ["paged_scores", "paged_select"]
    dsa.dsa_paged_index_topk(cache, batch, torch.empty(0, 4, DI, dtype=torch.bfloat16, device=DEV),
                             torch.empty(0, 4, device=DEV), 8)
    assert dsa.last_kernel_config()["kernels"] == []


def test_refusals_of_the_binding():
    m = Model([2], [30], 16, seed=71)
    cache, batch = m.to_gpu(dsa)
    q, w = index_inputs(m, 4)
    q, w = q.to(DEV), w.to(DEV)
    with pytest.raises(TypeError):
        dsa.dsa_paged_index_topk(cache, batch, q.float(), w, 8)
    with pytest.raises(ValueError):
        dsa.dsa_paged_index_topk(cache, batch, q, w[:1], 8)
    with pytest.raises(ValueError):
        dsa.dsa_paged_index_topk(cache, batch, q.cpu(), w, 8)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_paged_index_topk(cache, batch, q, w, 4096)
    assert e.value.status == dsa.DSA_ERR_UNSUPPORTED
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_paged_index_topk(cache, batch, q, w, 8, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == dsa.DSA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        dsa.PagedCache(cache.k, cache.v[:, :8], cache.k_idx, cache.khat)
    with pytest.raises(ValueError):
        dsa.PagedCache(cache.k.transpose(0, 1), cache.v, cache.k_idx, cache.khat)
    with pytest.raises(ValueError):
        dsa.PagedBatch(batch.block_table, batch.seq_lens, i32([0]))
    with pytest.raises(ValueError):
        dsa.dsa_cache_append(cache, batch, *[torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
                                             for n, d in ((2, D), (3, D), (2, DI))])
    with pytest.raises(dsa.DsaError) as e:  # rows 260 elements apart: not a multiple of 8
        x = torch.zeros(2, 260, dtype=torch.bfloat16, device=DEV)
        dsa.dsa_cache_append(cache, batch, x[:, :D], x[:, :D], x[:, :DI])
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG
    with pytest.raises(dsa.DsaError) as e:  # 12 tokens a page
        z = [torch.zeros(4, n, d, dtype=torch.bfloat16, device=DEV) for n, d in ((12, D), (12, D), (12, DI), (3, D))]
        dsa.dsa_cache_copy_pages(dsa.PagedCache(*z), i32([0]), i32([1]))
    assert e.value.status == dsa.DSA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        dsa.dsa_cache_compact(cache, dsa.PageTable(batch.block_table, batch.seq_lens, i32([1] * (cache.num_pages + 1))))
