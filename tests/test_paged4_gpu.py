"""The layer over a paged cache with keys and values in 4 bits on the GPU, against plain models in 64-bit CPU arithmetic."""
import math

import numpy as np
import pytest

from tests import _four as f4
from tests._paged import D, DI, HQ, random_selection
from tests.test_paged_gpu import LAYOUTS, Pages, check_topk, index_inputs, same_bits
from tests.test_rope_gpu import KINDS, bf16, check_queries, gpu, i32, queries, reported

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_context_sparse_index_gb300 as dsa
DEV = "cuda"


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def buffers(cache):
    return [cache.kv, cache.k_idx, cache.khat]


def check_cache4(cache, m):
    for n in ("kv", "k_idx", "khat"):
        assert same_bytes(getattr(cache, n).cpu(), getattr(m, n)), n


# --------------------------------------------------------------------------- writing and reading

@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", KINDS)
def test_append_bit_exact(layout, page, kind):
    """Codes and scales are the nearest ones of the turned keys and of the values; all other bytes stay."""
    m = f4.Model4(*LAYOUTS[layout], page, seed=1)
    ropes = f4.Turned(*KINDS[kind], 200)
    cache, batch = m.to_gpu4(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    given = queries(m, kind, m.T)
    r, ri = ropes.to_gpu(dsa)
    got = dsa.dsa_cache4_append(cache, batch, *gpu(k, v, ki), r, ri, *gpu(*given))
    kk, vv = dsa.dsa_cache4_read(cache, batch, m.T)
    dsa.dsa_sync_status()
    m.append4(k, v, ki, ropes)
    check_cache4(cache, m)
    check_queries(m, ropes, given, got)
    at = torch.tensor([m.slot(b, i) for _, b, i in m.rows()])
    assert same_bits(kk.cpu(), m.k.view(-1, D)[at]) and same_bits(vv.cpu(), m.v.view(-1, D)[at])


@pytest.mark.parametrize("new", [[1020, 4], [1021, 4], [700, 0, 1, 933, 2]])
def test_append_of_many_rows(new):
    m = f4.Model4(new, [61, 3, 2, 0, 5][:len(new)], 32, seed=2, pages_apart=72)
    ropes = f4.Turned(96, 48, False, 1200)
    cache, batch = m.to_gpu4(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    r, ri = ropes.to_gpu(dsa)
    dsa.dsa_cache4_append(cache, batch, *gpu(k, v, ki), r, ri)
    dsa.dsa_sync_status()
    m.append4(k, v, ki, ropes)
    check_cache4(cache, m)


def test_append_of_every_magnitude():
    """From what is too small for a scale to what saturates, zeros and negative zeros, ties of codes and of scales, a
    single large element among small ones."""
    n = 256
    m = f4.Model4([n], [0], 64, seed=3)
    cache, batch = m.to_gpu4(dsa)
    g = torch.Generator().manual_seed(4)
    k = (torch.randn(n, D, generator=g) * 2.0 ** (torch.arange(n)[:, None] / 4 - 40)).to(torch.bfloat16)
    v = torch.randint(-12, 13, (n, D), generator=g).float() / 2 * 2.0 ** torch.randint(-20, 12, (n, 8), generator=g).repeat_interleave(16, 1)
    v = v.to(torch.bfloat16)
    v[:40:2, ::16] = 6.0 * 2.0 ** torch.arange(-10, 10)[:, None]  # a scale that is a power of two: its codes meet all ties
    v[1] = 0.0
    v[3] = -0.0
    k[5] = 2.0 ** -133  # a subnormal number
    k[7, 3] = 3e38
    mids = 6 / 16 * (1 + (2 * torch.arange(8) + 1) / 16) * 2.0 ** torch.arange(-5, 11).view(-1, 1)  # between two scales
    k[9:25, ::16] = mids.to(torch.bfloat16)
    assert torch.equal(mids.to(torch.bfloat16).float(), mids.float())
    k[9:25, 1::16] = k[9:25, ::16] / 2
    dsa.dsa_cache4_append(cache, batch, *gpu(k, v, m.fill(n, DI)))
    kk, vv = dsa.dsa_cache4_read(cache, batch, n)
    dsa.dsa_sync_status()
    for x, y in ((k, kk), (v, vv)):
        want = f4.stands_for(*f4.quantise(x))
        assert torch.equal(y.cpu().double(), want)
    assert kk[7].max().item() == 3840 and torch.all(kk[5] == 0)


def test_append_of_infinities_and_nan():
    """Their groups stand for NaN, the others for what they held."""
    m = f4.Model4([4], [2], 16, seed=5)
    cache, batch = m.to_gpu4(dsa)
    k, v = m.fill(4, D), m.fill(4, D)
    k[1, 5], k[2, 127], v[2, 16], v[3, 15] = math.inf, -math.inf, math.nan, math.inf
    dsa.dsa_cache4_append(cache, batch, *gpu(k, v, m.fill(4, DI)))
    kk, vv = dsa.dsa_cache4_read(cache, batch, 4)
    dsa.dsa_sync_status()
    for x, y in ((k, kk), (v, vv)):
        torch.testing.assert_close(y.cpu().double(), f4.stands_for(*f4.quantise(x)), rtol=0, atol=0, equal_nan=True)
        assert torch.isnan(y).sum() == 32


def test_read_of_every_scale_and_code():
    """All bytes that an append may write stand for what the format says, wherever they lie."""
    pages, page = 16, 64
    cache = dsa.PagedCache4.empty(pages, page)
    g = torch.Generator().manual_seed(6)
    kv = torch.randint(0, 256, (pages * page // 4, 576), generator=g, dtype=torch.uint8)
    kv[:, 512:] = torch.randint(0, 0xE3, (pages * page // 4, 64), generator=g, dtype=torch.uint8)
    cache.kv.view(-1, 576).copy_(kv)
    n = pages * page
    batch = dsa.PagedBatch(i32(range(pages)).view(1, -1), i32([n]), i32([0, n]))
    wide = torch.full((n + 3, 2 * D + 8), 4.0, dtype=torch.bfloat16, device=DEV)
    k, v = dsa.dsa_cache4_read(cache, batch, n + 3, k=wide[:, :D], v=wide[:, D + 8:])
    dsa.dsa_sync_status()
    for p in range(0, n // 4, 3):
        kk, vv = f4.read(kv[p])
        assert torch.equal(k[4 * p:4 * p + 4].cpu().double(), kk) and torch.equal(v[4 * p:4 * p + 4].cpu().double(), vv)
    assert torch.all(wide[n:] == 4.0) and torch.all(wide[:, D:D + 8] == 4.0)  # padding rows, and between


def test_append_again_after_a_rejected_draft():
    """Tokens written again at earlier positions replace their own bytes of a pool, and no others."""
    m = f4.Model4([7], [6], 16, seed=7)
    ropes = f4.Turned(64, 64, False, 20)
    cache, batch = m.to_gpu4(dsa)
    r, ri = ropes.to_gpu(dsa)
    draft = [m.fill(7, d) for d in (D, D, DI)]
    dsa.dsa_cache4_append(cache, batch, *gpu(*draft), r, ri)
    m.append4(*draft, ropes)
    m.new, m.lens, m.cu, m.T, m.old = [3], [11], [0, 3], 3, [8]
    again = [m.fill(3, d) for d in (D, D, DI)]
    batch = dsa.PagedBatch(m.table.to(DEV), i32([11]), i32([0, 3]))
    dsa.dsa_cache4_append(cache, batch, *gpu(*again), r, ri)
    dsa.dsa_sync_status()
    m.append4(*again, ropes)
    check_cache4(cache, m)


# --------------------------------------------------------------------------- pages and the indexer

def random_cache4(num_pages, page, seed=5, apart=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def new(n, d, dtype):
        x = torch.randint(0, 256, (num_pages, n * d * dtype.itemsize + 2 * apart), generator=g, device=DEV, dtype=torch.uint8)
        return x.view(dtype).as_strided((num_pages, n, d), (n * d + 2 * apart // dtype.itemsize, d, 1))
    return dsa.PagedCache4(new(page // 4, 576, torch.uint8), new(page, DI, torch.bfloat16), new(page // 4, D, torch.bfloat16))


@pytest.mark.parametrize("page,apart", [(16, 0), (64, 40), (256, 0), (1024, 8)])
def test_copy_pages(page, apart):
    caches = [random_cache4(11, page, seed=s, apart=apart) for s in range(3)]
    want = [[b.clone() for b in buffers(c)] for c in caches]
    src, dst = [3, 3, 0, 10, 7], [1, 4, 2, 9, 7]
    dsa.dsa_cache_copy_pages(caches, i32(src), i32(dst))
    dsa.dsa_sync_status()
    for c, w in zip(caches, want):
        for b, x in zip(buffers(c), w):
            x[dst] = x[src]
            assert same_bytes(b, x)
    reported(lambda: dsa.dsa_cache_copy_pages(caches[0], i32([0, 11]), i32([2, 1])))


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("layers", [1, 34])
def test_forks_frees_and_compaction(page, layers):
    """Every layer's pages move alike, as the plain bookkeeping says."""
    p = Pages([40, 2 * page + 3, 0, 0, 0, page, 7], page, 30, 6, seed=layers)
    t = p.to_gpu()
    caches = [random_cache4(30, page, seed=s) for s in range(layers)]
    want = [[b.clone() for b in buffers(c)] for c in caches]
    arg = caches[0] if layers == 1 else caches

    def check(moves):
        for c, w in zip(caches, want):
            for b, x in zip(buffers(c), w):
                for s, d in moves:
                    x[d] = x[s]
                assert same_bytes(b, x)
        p.check(t)

    n, moves = p.fork([0, 1, 1], [2, 3, 4])
    assert dsa.dsa_cache_fork(arg, t, i32([0, 1, 1]), i32([2, 3, 4])).item() == n
    check(moves)
    p.free([1, 5])
    dsa.dsa_cache_free(arg, t, i32([1, 5]))
    used, moves = p.compact()
    assert dsa.dsa_cache_compact(arg, t).tolist() == [used, len(moves)]
    dsa.dsa_sync_status()
    check(moves)
    assert dsa.dsa_cache_reserve(arg, t, i32([1] * 7)).item() == p.reserve([1] * 7)
    check([])


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 7, 11], [40, 3, 1]])
def test_index_is_that_of_the_bf16_cache(new):
    m = f4.Model4(new, [1200, 37, 517], 32, seed=8, ints=True, pages_apart=24)
    cache, batch = m.to_gpu4(dsa)
    q, w = index_inputs(m, 8)
    got = dsa.dsa_paged_index_topk(cache, batch, q.to(DEV), w.to(DEV), 30)
    assert dsa.last_kernel_config()["entry"] == "dsa_paged4_index_topk"
    dsa.dsa_sync_status()
    check_topk(m, q, w, 30, got)
    same, _ = m.to_gpu(dsa)
    assert torch.equal(got, dsa.dsa_paged_index_topk(same, batch, q.to(DEV), w.to(DEV), 30))


# --------------------------------------------------------------------------- attention

def check_attention4(m, q, sel, scale, o, lse, rows=None):
    ro, rl, av, mag = m.attention(q, sel, scale)
    bo, bl = f4.attention4_bounds(ro, av, rl, mag, *m.abs_values(sel))
    rows = slice(0, m.T) if rows is None else rows
    err = (o.cpu().double()[:m.T] - ro).abs()[rows]
    assert torch.all(err <= bo[rows]), (err / bo[rows]).max()
    err = (lse.cpu().double()[:m.T] - rl).abs()[rows]
    assert torch.all(err <= bl[rows]), (err / bl[rows]).max()


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("topk", [1, 15, 16, 64])
def test_attention_small(layout, page, topk):
    m = f4.Model4(*LAYOUTS[layout], page, seed=31)
    cache, batch = m.to_gpu4(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, topk, seed=1)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)


def test_attention_picks_single_tokens_and_dimensions():
    """A key that one query meets alone gives its value back: every place of a pool, every dimension, every head."""
    n = 64
    m = f4.Model4([1] * 4, [n - 4 + j for j in range(4)], 64, seed=32)
    cache, batch = m.to_gpu4(dsa)
    sel = torch.full((4, 15), -1, dtype=torch.int32)
    sel[:] = torch.arange(15)
    k = m.k.view(-1, D).double()
    for trial in range(8):
        q = torch.zeros(4, HQ, D, dtype=torch.bfloat16)
        aim = torch.randint(0, n - 4, (4, HQ), generator=torch.Generator().manual_seed(trial))
        for r in range(4):
            for h in range(HQ):
                q[r, h] = k[m.slot(r, int(aim[r, h]))].to(torch.bfloat16) * 64
        o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
        dsa.dsa_sync_status()
        check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)
        for r in range(4):  # the aim's logit is ahead of all others by more than 40: its value alone
            slots = [m.slot(r, t) for t in range(n - 4 + r + 1)]
            first = (q[r].double() @ k[slots].T / math.sqrt(D)).topk(2, dim=1)
            sure = first.values[:, 0] - first.values[:, 1] > 40
            want = m.v.view(-1, D)[torch.tensor(slots)[first.indices[:, 0]]]
            assert torch.equal(o[r].cpu()[sure], want[sure]) and sure.any()  # (a sum that ends in -0 is +0)


@pytest.mark.parametrize("rows", [1, 2, 14, 16, 25, 38, 57, 60, 76, 100, 152, 153, 228, 229, 400])
@pytest.mark.parametrize("topk", [512, 300, 96, 80])
def test_attention_every_split(rows, topk):
    """Every number of CTAs per row; rows that keep fewer pools than the others leave CTAs without keys."""
    m = f4.Model4([1] * rows, [50 + 37 * j % 3000 for j in range(rows)], 64, seed=37)
    cache, batch = m.to_gpu4(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, topk, seed=rows, fewer=True)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    o2, lse2 = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    assert same_bits(o, o2) and torch.equal(lse, lse2)
    check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("new,old,topk", [([1], [9000], 2048), ([3], [70000], 1000), ([200], [8200], 2048),
                                          ([19], [8300], 2048), ([60], [9000], 1500)])
def test_attention_long(new, old, topk):
    m = f4.Model4(new, old, 128, seed=41, pages_apart=24)
    cache, batch = m.to_gpu4(dsa)
    q, sel = m.fill(m.T, HQ, D) * 2, random_selection(m, topk, seed=2)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), scale=0.1)
    dsa.dsa_sync_status()
    check_attention4(m, q, sel, 0.1, o, lse)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("power", [-126, -60, -20, 20, 60, 110])
def test_attention_of_queries_of_any_magnitude(rows, power):
    """Queries far outside of fp16's range, each head with its own, and a head of zeros; the scale brings the logits
    back."""
    m = f4.Model4([1] * rows, [90 + j for j in range(rows)], 16, seed=42)
    cache, batch = m.to_gpu4(dsa)
    q = m.fill(m.T, HQ, D)
    q[:, 3] = 0
    q[:, 4] = (q[:, 4].float() * 2.0 ** -12).to(torch.bfloat16)
    q[:, 5] = (q[:, 5].float() * 2.0 ** -(torch.arange(D) % 24)).to(torch.bfloat16)
    q = (q.double() * 2.0 ** power).to(torch.bfloat16)
    sel, scale = random_selection(m, 20, seed=3), 2.0 ** -power / math.sqrt(D)
    scale = min(scale, 2.0 ** 120)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), scale=scale)
    dsa.dsa_sync_status()
    check_attention4(m, q, sel, scale, o, lse)


def huge_bounds(o, av, lse, sum_v, keys):
    """What the arithmetic may be off by where the products are exact: integers whose sums have at most 24 bits.  A weight's
    exponent is a difference of products times a factor (a rounding each, two in the factor: 2^-22 of an exponent below 64
    that counts at all, which makes 2^-16 of the weight), taken at most three times (warp, CTA, cluster) with 2^-21 for each
    exponential: below 2^-14 in all, and for the normaliser as much.  P is rounded to fp16: 2^-11 of it, or 2^-25 where it
    is subnormal, and the normaliser is at least 1.  Sums of n terms, twice, and o rounded once more.  lse: a product, a
    sum and a product with rounded constants, six roundings of 2^-24 each."""
    n = keys[:, None] * 2.0 ** -23
    rel = 2.0 ** -13 + 2.0 ** -11 + n
    off = rel[..., None] * av + 2.0 ** -25 * sum_v[:, None] + 1e-30
    return off + 2.0 ** -8 * (o.abs() + off), 2.0 ** -13 + n + 2.0 ** -21 * lse.abs()


# (products reach some 150: logits of 2^7 to 2^107)
POWERS = [0, 4, 10, 17, 20, 21, 22, 23, 25, 27, 30, 53, 100]


@pytest.mark.parametrize("rows,old,topk", [(3, 1020, 200), (40, 700, 120), (100, 200, 50), (300, 200, 40), (500, 60, 12)])
@pytest.mark.parametrize("power", POWERS)
def test_attention_of_huge_logits(rows, old, topk, power):
    """Exact products and any finite logits: the largest one's weight is one, whatever its logit's last bit stands for."""
    m = f4.Model4([1] * rows, [old + j % 50 for j in range(rows)], 16, seed=61, ints=True)
    cache, batch = m.to_gpu4(dsa)
    q, sel, scale = m.fill(m.T, HQ, D), random_selection(m, topk, seed=6), 2.0 ** power
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), scale=scale)
    dsa.dsa_sync_status()
    ro, rl, av, _ = m.attention(q, sel, scale)
    bo, bl = huge_bounds(ro, av, rl, *m.abs_values(sel))
    err = (o.cpu().double() - ro).abs()
    assert torch.all(err <= bo), (err / bo).max()
    err = (lse.cpu().double() - rl).abs()
    assert torch.all(err <= bl), (err / bl).max()


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("power", POWERS)
def test_weights_of_huge_logits_sum_to_one(rows, power):
    """Products of any numbers, and values that are all 3: so is every output (the weights' sum and the normaliser agree to
    2^-11, and bf16's neighbours of 3 are 2^-6 away)."""
    m = f4.Model4([1] * rows, [300 + j % 50 for j in range(rows)], 16, seed=62)
    flat = m.kv.view(-1, 576)
    for t in range(4):
        _, code, _, scale = f4.places(t)
        flat[:, code], flat[:, scale] = 0x77, 0x90  # 6 times 8 / 16
    assert torch.all(f4.read(flat[0])[1] == 3)
    cache, batch = m.to_gpu4(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, 60, seed=7)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), scale=2.0 ** power)
    dsa.dsa_sync_status()
    assert torch.all(o == 3) and torch.isfinite(lse).all()


def test_attention_records_how_a_row_is_split():
    """Every number of CTAs a row has, and both lengths of the ring, among the sizes of a device of any width."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    met = set()
    for topk in (512, 96):
        for rows in sorted({1, sms // 12, sms // 6, sms // 4, sms * 3 // 8, sms // 2, sms * 2 // 3, sms, sms * 3 // 2, sms * 2,
                            sms * 3, sms * 3 + 1}):
            m = f4.Model4([1] * rows, [50] * rows, 16, seed=63)
            cache, batch = m.to_gpu4(dsa)
            sel = torch.full((rows, topk), -1, dtype=torch.int32)
            dsa.dsa_paged4_sparse_attn_fwd(cache, batch, m.fill(rows, HQ, D).to(DEV), sel.to(DEV))
            c = dsa.last_kernel_config()
            ctas, ring = c["params"]["ctas_per_row"], c["params"]["ring_blocks"]
            assert ("cluster" in c["variant"]) == (ctas > 1) and (ring == 6 or rows > 3 * sms)
            met.add((ctas, ring))
    dsa.dsa_sync_status()
    assert met == {(8, 6), (6, 6), (4, 6), (2, 6), (1, 6), (1, 4)}


@pytest.mark.parametrize("rows", [3, 100, 500])
def test_attention_reads_nothing_it_does_not_attend_to(rows):
    """NaN in every slot that no row attends to, positions behind the last token among them."""
    m = f4.Model4([1] * rows, [40 + 3 * j for j in range(rows)], 16, seed=43)
    sel = random_selection(m, 8, seed=3)
    seen = torch.zeros(m.pages * m.page, dtype=torch.bool)
    for r, b, i in m.rows():
        for t in [4 * p + e for p in sel[r].tolist() if p >= 0 for e in range(4)] + list(range(i // 4 * 4, i + 1)):
            seen[m.slot(b, t)] = True
    for t in range(4):
        at = torch.nonzero(~seen.view(-1, 4)[:, t])[:, 0]
        for place in f4.places(t)[2:]:
            m.kv.view(-1, 576)[at[:, None], place] = 0xFF
        for place in f4.places(t)[:2]:
            m.kv.view(-1, 576)[at[:, None], place] = 0x77
    cache, batch = m.to_gpu4(dsa)
    q = m.fill(m.T, HQ, D)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)


def test_attention_of_nan_and_infinite_inputs():
    """A NaN that is attended to reaches its heads' outputs (of a value: its group's), and no other row's."""
    m = f4.Model4([1] * 3, [100] * 3, 16, seed=44)
    q, sel = m.fill(3, HQ, D), random_selection(m, 10, seed=5)
    s = m.slot(1, 4 * int(sel[1, 3]) + 2)
    for place in f4.places(s % 4)[3:]:
        m.kv.view(-1, 576)[s // 4, place[5]] = 0xFF  # the group of dimensions 80..95 of a value
    cache, batch = m.to_gpu4(dsa)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    assert torch.isnan(o[1, :, 80:96]).all() and torch.isfinite(o[1, :, :80]).all() and torch.isfinite(o[[0, 2]]).all()
    assert torch.isfinite(lse).all()
    q[2, 7, 9], q[0, 2, 0] = math.nan, math.inf
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))
    dsa.dsa_sync_status()
    assert torch.isnan(o[2, 7]).all() and torch.isnan(lse[2, 7]) and torch.isfinite(lse[2, 8])
    assert not torch.isfinite(lse[0, 2]) and torch.isfinite(o[0, 3]).all()


@pytest.mark.parametrize("rows", [2, 200])
def test_attention_leaves_padding_and_given_outputs(rows):
    m = f4.Model4([1] * rows, [100] * rows, 32, seed=47)
    cache, batch = m.to_gpu4(dsa)
    q = m.fill(m.T + 5, HQ, D)
    sel = torch.cat([random_selection(m, 16, seed=4), torch.zeros(5, 16, dtype=torch.int32)])
    o = torch.full((m.T + 5, HQ, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((m.T + 5, HQ), 5.0, device=DEV)
    dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV), o=o, lse=lse)
    dsa.dsa_sync_status()
    assert torch.all(o[m.T:] == 3.0) and torch.all(lse[m.T:] == 5.0)
    check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("what", ["page", "page_high", "length", "offsets", "selection", "order"])
@pytest.mark.parametrize("rows", [4, 300])
def test_what_is_out_of_range_is_reported_and_not_followed(what, rows):
    m = f4.Model4([1] * rows, [200 + j % 50 for j in range(rows)], 16, seed=53)
    good = f4.Model4([1] * rows, [200 + j % 50 for j in range(rows)], 16, seed=53)
    bad = 2
    sel, q = random_selection(m, 16, seed=5), m.fill(m.T, HQ, D)
    if what in ("page", "page_high"):
        m.table[bad, int(sel[bad, 0]) // 4] = -1 if what == "page" else m.pages
    elif what == "length":
        m.lens[bad] = m.width * 16 + 1
    elif what == "offsets":
        m.lens[bad] = 0
    elif what == "selection":
        sel[bad, 15] = (m.lens[bad] - 1) // 4
    else:
        sel[bad, 1] = sel[bad, 0]
    cache, batch = m.to_gpu4(dsa)
    out = []
    reported(lambda: out.extend(dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q.to(DEV), sel.to(DEV))))
    ok = [r for r in range(rows) if r != bad]
    sel[bad] = -1
    check_attention4(good, q, sel, 1 / math.sqrt(D), *out, rows=ok)
    if what in ("page", "page_high", "length", "offsets"):  # appending and reading follow the same numbers
        if what in ("page", "page_high"):
            m.table[bad] = -1 if what == "page" else m.pages
            batch.block_table.copy_(m.table)
        kk = torch.full((m.T, D), 9.0, dtype=torch.bfloat16, device=DEV)
        reported(lambda: dsa.dsa_cache4_read(cache, batch, m.T, k=kk))
        assert torch.all(kk[bad] == 9.0)
        new = [m.fill(m.T, d) for d in (D, D, DI)]
        before = cache.kv.clone()
        reported(lambda: dsa.dsa_cache4_append(cache, batch, *gpu(*new)))
        s = good.slot(bad, good.lens[bad] - 1) // 4
        assert torch.equal(cache.kv.view(-1, 576)[s], before.view(-1, 576)[s])


def test_large_cache_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of the 4-bit buffer are written, read, attended to and copied."""
    page, pages = 1024, 31000  # kv: 4.6 GB
    cache = dsa.PagedCache4.empty(pages, page)
    n = 3 * page + 5
    batch = dsa.PagedBatch(i32([pages - 1, 0, pages - 2, 1]).view(1, 4), i32([n]), i32([0, n]))
    near = dsa.PagedCache4.empty(4, page)
    near_batch = dsa.PagedBatch(i32([0, 1, 2, 3]).view(1, 4), i32([n]), i32([0, n]))
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(n, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    ki = torch.randint(-3, 4, (n, DI), generator=g, device=DEV).to(torch.bfloat16)
    dsa.dsa_cache4_append(cache, batch, k, v, ki)
    dsa.dsa_cache4_append(near, near_batch, k, v, ki)
    for a, b in zip(dsa.dsa_cache4_read(cache, batch, n), dsa.dsa_cache4_read(near, near_batch, n)):
        assert same_bits(a, b)
    assert torch.equal(cache.kv[pages - 2], near.kv[2])
    qi = torch.randint(-3, 4, (n, 4, DI), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randint(0, 4, (n, 4), generator=g, device=DEV).float()
    sel = dsa.dsa_paged_index_topk(cache, batch, qi, w, 64)
    assert torch.equal(sel, dsa.dsa_index_topk(qi, ki, w, chunk=256, topk=64))
    q = torch.randn(n, HQ, D, generator=g, device=DEV).to(torch.bfloat16)
    for a, b in zip(dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q, sel),
                    dsa.dsa_paged4_sparse_attn_fwd(near, near_batch, q, sel)):
        assert torch.equal(a, b)
    dsa.dsa_cache_copy_pages(cache, i32([pages - 1]), i32([pages - 3]))
    dsa.dsa_sync_status()
    assert torch.equal(cache.kv[pages - 3], near.kv[0])


# --------------------------------------------------------------------------- as they are used together

def test_attention_is_that_of_the_contiguous_call_on_what_the_cache_holds():
    """Append (turned), read back, and the training forward on the read rows: the same layer up to the bf16 rounding of
    the weights there (2^-8 of each) and both outputs' rounding."""
    S = 500
    m = f4.Model4([S], [0], 64, seed=61)
    ropes = f4.Turned(128, 64, False, S)
    cache, batch = m.to_gpu4(dsa)
    r, ri = ropes.to_gpu(dsa)
    new = gpu(m.fill(S, D), m.fill(S, D), m.fill(S, DI))
    q, _ = dsa.dsa_cache4_append(cache, batch, *new, r, ri, q=m.fill(S, HQ, D).to(DEV))
    sel = random_selection(m, 20, seed=7).to(DEV)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q, sel)
    k, v = dsa.dsa_cache4_read(cache, batch, S)
    wo, wl = dsa.dsa_sparse_attn_fwd(q, k, v, sel)
    dsa.dsa_sync_status()
    torch.testing.assert_close(o.float(), wo.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    torch.testing.assert_close(lse, wl, rtol=1e-5, atol=1e-5)


def test_prompts_in_chunks_then_tokens_with_forks_and_compaction():
    """As a server runs it: prompts in chunks, tokens, drafts that are rejected, forks, a compaction; each step's outputs
    are the 64-bit model's on the tokens so far, turned and quantised."""
    page, topk, Hi = 16, 12, 4
    cache = random_cache4(120, page)
    t = dsa.PageTable.empty(cache, max_seqs=4, max_pages=20)
    ropes = f4.Turned(64, 32, True, 400)
    r, ri = ropes.to_gpu(dsa)
    g = torch.Generator().manual_seed(3)
    hist = {s: [torch.zeros(0, D), torch.zeros(0, D)] for s in range(4)}
    scale = 1 / math.sqrt(D)

    def step(adds):
        add = [adds.get(s, 0) for s in range(4)]
        taken = dsa.dsa_cache_reserve(cache, t, i32(add))
        T = sum(add)
        k, v, ki = (torch.randn(T, d, generator=g).to(torch.bfloat16) for d in (D, D, DI))
        q, qi = torch.randn(T, HQ, D, generator=g).to(torch.bfloat16), torch.randn(T, Hi, DI, generator=g).to(torch.bfloat16)
        w = torch.rand(T, Hi, generator=g)
        batch = dsa.PagedBatch(t.block_table, t.seq_lens, i32(np.concatenate([[0], np.cumsum(add)])))
        qr, qir = dsa.dsa_cache4_append(cache, batch, *gpu(k, v, ki), r, ri, *gpu(q, qi), reserved=taken)
        sel = dsa.dsa_paged_index_topk(cache, batch, qir, w.to(DEV), topk)
        o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, qr, sel)
        kk, vv = dsa.dsa_cache4_read(cache, batch, T)
        dsa.dsa_sync_status()
        sel, o, lse, qr, at = sel.cpu(), o.cpu().double(), lse.cpu().double(), qr.cpu().double(), 0
        for s, n in enumerate(add):
            old = hist[s][0].shape[0]
            pos = torch.arange(old, old + n)
            mine = slice(at, at + n)
            want_k = f4.stands_for(*f4.quantise(f4.turned_key(k[mine], ropes.k[pos], True))) if n else torch.zeros(0, D)
            want_v = f4.stands_for(*f4.quantise(v[mine])) if n else torch.zeros(0, D)
            assert torch.equal(kk[mine].cpu().double(), want_k.double()) and torch.equal(vv[mine].cpu().double(), want_v.double())
            hist[s] = [torch.cat([a.double(), b.double()]) for a, b in zip(hist[s], (want_k, want_v))]
            for j in range(n):
                i = old + j
                toks = [4 * p + e for p in sel[at + j].tolist() if p >= 0 for e in range(4)] + list(range(i // 4 * 4, i + 1))
                assert len([p for p in sel[at + j].tolist() if p >= 0]) == min(topk, i // 4)
                x = qr[at + j] @ hist[s][0][toks].T * scale
                torch.testing.assert_close(lse[at + j], torch.logsumexp(x, 1), rtol=1e-5, atol=1e-5)
                want = torch.softmax(x, 1) @ hist[s][1][toks]
                torch.testing.assert_close(o[at + j], want, rtol=2.0 ** -7, atol=2.0 ** -8)
            at += n

    step({0: 50, 1: 3})
    step({0: 61, 1: 17})
    for _ in range(3):
        step({0: 1, 1: 1})
    step({0: 5, 1: 4})  # drafts, of which some are rejected
    dsa.dsa_cache_reserve(cache, t, i32([-3, -4, 0, 0]))
    hist[0], hist[1] = [x[:-3] for x in hist[0]], [x[:-4] for x in hist[1]]
    step({0: 1, 1: 2})
    dsa.dsa_cache_fork(cache, t, i32([0, 0]), i32([2, 3]))
    hist[2] = hist[3] = hist[0]
    for _ in range(5):
        step({0: 1, 1: 1, 2: 1, 3: 1})
    dsa.dsa_cache_free(cache, t, i32([0, 1]))
    hist[0] = hist[1] = [torch.zeros(0, D), torch.zeros(0, D)]
    dsa.dsa_cache_compact(cache, t)
    for _ in range(3):
        step({2: 1, 3: 2})
    step({0: 30, 2: 5, 3: 1})


def test_decoding_step_in_a_replayed_graph():
    """reserve, append with queries, indexer, attention and reading back captured once and replayed with new tokens and
    growing lengths: what eager calls give on a copy of the cache."""
    page, B, Hi, topk = 16, 3, 4, 8
    m = f4.Model4([1] * B, [40, 9, 60], page, seed=71, width_extra=6, spare=24)
    ropes = f4.Turned(128, 64, False, 200)
    r, ri = ropes.to_gpu(dsa)

    def world():
        cache, _ = m.to_gpu4(dsa)
        count = torch.zeros(m.pages, dtype=torch.int32)
        count[m.table[m.table >= 0].long()] = 1
        t = dsa.PageTable(m.table.to(DEV), i32([n - 1 for n in m.lens]), count.to(DEV))
        return cache, t, dsa.PagedBatch(t.block_table, t.seq_lens, i32(range(B + 1)))

    def step(w, x):
        cache, t, batch = w
        taken = dsa.dsa_cache_reserve(cache, t, x["add"])
        q, qi = dsa.dsa_cache4_append(cache, batch, x["k"], x["v"], x["ki"], r, ri, x["q"], x["qi"], reserved=taken)
        sel = dsa.dsa_paged_index_topk(cache, batch, qi, x["w"], topk)
        return [taken, sel, q, *dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q, sel), *dsa.dsa_cache4_read(cache, batch, B)]

    def tokens(seed):
        return {"add": i32([1] * B), "k": bf16(B, D, seed=seed).to(DEV), "v": bf16(B, D, seed=seed + 1).to(DEV),
                "ki": bf16(B, DI, seed=seed + 2).to(DEV), "q": bf16(B, HQ, D, seed=seed + 3).to(DEV),
                "qi": bf16(B, Hi, DI, seed=seed + 4).to(DEV), "w": bf16(B, Hi, seed=seed + 5).float().to(DEV)}

    a, b, x = world(), world(), tokens(0)
    step(world(), x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a, x)
    for n in range(12):
        new = tokens(10 * n)
        for name in x:
            x[name].copy_(new[name])
        graph.replay()
        for y, z in zip(out, step(b, new)):
            assert same_bytes(y, z)
    dsa.dsa_sync_status()
    for y, z in zip(buffers(a[0]), buffers(b[0])):
        assert same_bytes(y, z)


def test_calls_on_a_stream_of_their_own():
    m = f4.Model4([1, 40], [5000, 100], 64, seed=63)
    cache, batch = m.to_gpu4(dsa)
    q, sel = m.fill(m.T, HQ, D), random_selection(m, 64, seed=9)
    side = torch.cuda.Stream()
    qg, sg, new = q.to(DEV), sel.to(DEV), gpu(m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI))
    side.wait_stream(torch.cuda.current_stream())
    dsa.dsa_cache4_append(cache, batch, *new, stream=side)
    o, lse = dsa.dsa_paged4_sparse_attn_fwd(cache, batch, qg, sg, stream=side)
    k, _ = dsa.dsa_cache4_read(cache, batch, m.T, stream=side)
    side.synchronize()
    dsa.dsa_sync_status(side)
    m.append4(*[x.cpu() for x in new])
    check_attention4(m, q, sel, 1 / math.sqrt(D), o, lse)
    assert same_bits(k.cpu(), m.k.view(-1, D)[[m.slot(b, i) for _, b, i in m.rows()]])
