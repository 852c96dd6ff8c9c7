"""Rotated positions on the GPU, against plain 64-bit models: heads turned and turned back, appends that turn keys and
queries, and the layer trained with them."""
import ctypes
import gc
import math

import pytest

from tests import _four as f4
from tests._paged import D, DI, HQ
from tests._util import MAX_ABS, REL_L2
from tests.test_paged_gpu import LAYOUTS, check_cache, same_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_context_sparse_index_gb300 as dsa
DEV = "cuda"


def bf16(*shape, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def check_turned(got, x, cs, inter, inverse=False):
    ref, mag = f4.turn(x, cs, inter, inverse)
    err, bound = (got.cpu().double() - ref).abs(), f4.turn_bound(ref, mag)
    assert torch.all(err <= bound), (err / bound).max()
    assert same_bits(got.cpu()[..., cs.shape[-1]:], x[..., cs.shape[-1]:])  # what is not turned


def reported(call=lambda: None):
    call()
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_sync_status()
    assert e.value.status == dsa.DSA_ERR_INTERNAL
    dsa.dsa_clear_status()


# --------------------------------------------------------------------------- heads

@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,dims", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 80), (128, 96), (128, 112), (128, 128)])
@pytest.mark.parametrize("H", [1, 2, 3, 7, 16, 33, 128])
def test_rope(D, dims, H, inter):
    """Every lane mapping: one row a warp or several, heads that end inside a pass, halves that are no power of two."""
    S = 37
    cs = f4.table(S + 5, dims)
    x = bf16(S, H, D, seed=H)
    rope = dsa.Rope(cs.to(DEV), interleaved=inter)
    for inverse in (False, True):
        got = dsa.dsa_rope(x.to(DEV), rope, q_begin=5, inverse=inverse)
        dsa.dsa_sync_status()
        check_turned(got, x, cs[5:], inter, inverse)


@pytest.mark.parametrize("S", [1, 2, 255, 4099])
def test_rope_by_given_positions(S):
    """A packed batch, the same position more than once, the table's first and last row; positions in any order."""
    cs = f4.table(600, 64)
    pos = torch.randint(0, 600, (S,), generator=torch.Generator().manual_seed(S))
    pos[0] = 599
    pos[-1] = 0 if S > 1 else 599
    for H, d, inter in ((16, 128, False), (1, 64, True)):
        x = bf16(S, H, d, seed=S)
        got = dsa.dsa_rope(x.to(DEV), dsa.Rope(cs.to(DEV), interleaved=inter), positions=pos.int().to(DEV))
        dsa.dsa_sync_status()
        check_turned(got, x, cs[pos], inter)


def test_rope_of_one_head_a_row_in_place_and_strided():
    """[S, D] tensors, out of a fused projection, into a strided output, and onto themselves; nothing else is written."""
    S, cs = 133, f4.table(200, 96)
    wide = bf16(S, 8 + D + 24, seed=2)
    rope = dsa.Rope(cs.to(DEV))
    gpu = wide.to(DEV)
    check_turned(dsa.dsa_rope(gpu[:, 8:8 + D], rope)[:, None], wide[:, None, 8:8 + D], cs[:S], False)
    out = torch.full((S, 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    got = dsa.dsa_rope(gpu[:, 8:8 + D], rope, out=out[:, 1])
    check_turned(got[:, None], wide[:, None, 8:8 + D], cs[:S], False)
    assert torch.all(out[:, 0] == 7) and torch.all(out[:, 2] == 7)
    dsa.dsa_rope(gpu[:, 8:8 + D], rope, out=gpu[:, 8:8 + D])
    dsa.dsa_sync_status()
    check_turned(gpu[:, None, 8:8 + D], wide[:, None, 8:8 + D], cs[:S], False)
    assert same_bits(gpu[:, :8].cpu(), wide[:, :8]) and same_bits(gpu[:, 8 + D:].cpu(), wide[:, 8 + D:])
    heads = wide[:, 16:16 + D].reshape(S, 2, 64)  # two heads of a row that is wider, in place
    view = gpu.copy_(wide.to(DEV))[:, 16:16 + D].unflatten(1, (2, 64))
    narrow = f4.table(S, 32)
    dsa.dsa_rope(view, dsa.Rope(narrow.to(DEV), interleaved=True), out=view)
    check_turned(view, heads, narrow, True)


def test_rope_of_positions_that_the_table_does_not_have():
    x, cs = bf16(6, 4, 64), f4.table(10, 64)
    out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    pos = [0, 10, 3, -1, 9, 2 ** 31 - 1]
    reported(lambda: dsa.dsa_rope(x.to(DEV), dsa.Rope(cs.to(DEV)), positions=i32(pos), out=out))
    good = [0, 2, 4]
    check_turned(out[good], x[good], cs[torch.tensor(pos)[good]], False)
    assert torch.all(out[[1, 3, 5]] == 3.0)


def test_rope_of_nothing_and_of_a_strided_table():
    wide = torch.full((50, 72), math.nan)
    wide[:, 4:68] = f4.table(50, 64)
    rope = dsa.Rope(wide.to(DEV)[:, 4:68], interleaved=True)
    assert dsa.dsa_rope(torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), rope).shape == (0, 4, 64)
    x = bf16(50, 4, 64)
    check_turned(dsa.dsa_rope(x.to(DEV), rope), x, f4.table(50, 64), True)
    dsa.dsa_sync_status()


def test_rope_of_extreme_numbers():
    """Infinities and NaN stay where they are and reach their partners as the formula has it; subnormal results."""
    cs = torch.tensor([[0.625] * 8 + [0.75] * 8])
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    x[0, 0, :4] = torch.tensor([math.inf, math.nan, 3e38, 1e-39])
    x[0, 0, 8:12] = torch.tensor([1.0, 1.0, -3e38, 1e-39])
    got = dsa.dsa_rope(x.to(DEV), dsa.Rope(cs.to(DEV))).cpu()[0, 0].double()
    dsa.dsa_sync_status()
    assert got[0] == math.inf and got[8] == math.inf and torch.isnan(got[1]) and torch.isnan(got[9])
    assert got[2] == math.inf  # 4.1e38 is beyond bf16
    ref, mag = f4.turn(x, cs, False)
    bound = (f4.turn_bound(ref, mag) + 2.0 ** -149)[0, 0]
    for j in (3, 11):  # fp32 subnormals
        assert abs(got[j] - ref[0, 0, j]) <= bound[j] and got[j] != 0
    assert torch.all(got[16:] == 0)


@pytest.mark.parametrize("inter", [False, True])
def test_turning_back_is_the_adjoint(inter):
    """<dy, J x> = <J' dy, x>: both sides by the kernel, off by the roundings of their outputs (half a bf16 step each, and
    the fp32 sums')."""
    S, H, cs = 200, 16, f4.table(200, 128) * 1.25
    x, dy = bf16(S, H, D, seed=1), bf16(S, H, D, seed=2)
    rope = dsa.Rope(cs.to(DEV), interleaved=inter)
    y = dsa.dsa_rope(x.to(DEV), rope).cpu().double()
    dx = dsa.dsa_rope(dy.to(DEV), rope, inverse=True).cpu().double()
    dsa.dsa_sync_status()
    off = ((y * dy.double()).sum() - (dx * x.double()).sum()).abs()
    ey = f4.turn_bound(*f4.turn(x, cs, inter))
    ex = f4.turn_bound(*f4.turn(dy, cs, inter, inverse=True))
    assert off <= (ey * dy.double().abs()).sum() + (ex * x.double().abs()).sum()


def test_rope_at_large_sizes():
    """Offsets past 2^31 elements; sampled rows."""
    S, H = 1 << 20, 17  # 2.3e9 elements
    x = torch.empty(S, H, D, dtype=torch.bfloat16, device=DEV)
    for r in range(0, S, 1 << 17):
        x[r:r + (1 << 17)].normal_(generator=torch.Generator(device=DEV).manual_seed(r))
    cs = f4.table(S, 32, base=10000.0)
    rope = dsa.Rope(cs.to(DEV))
    at = torch.tensor([0, 1, 12345, S // 2, 986895, S - 2, S - 1])
    want = x[at.to(DEV)].cpu()
    dsa.dsa_rope(x, rope, out=x)
    dsa.dsa_sync_status()
    check_turned(x[at.to(DEV)], want, cs[at], False)


def test_rope_in_a_replayed_graph_and_on_another_stream():
    S, cs = 40, f4.table(100, 64)
    x, pos, rope = bf16(S, 4, 64).to(DEV), i32(range(S)), dsa.Rope(cs.to(DEV))
    out = torch.empty_like(x)
    dsa.dsa_rope(x, rope, positions=pos, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_rope(x, rope, positions=pos, out=out)
    for seed in (1, 2):
        new, at = bf16(S, 4, 64, seed=seed), torch.randperm(100, generator=torch.Generator().manual_seed(seed))[:S]
        x.copy_(new)
        pos.copy_(at.int())
        graph.replay()
        check_turned(out, new, cs[at], False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_rope(x, rope, q_begin=60, stream=side)
    side.synchronize()
    dsa.dsa_sync_status(side)
    check_turned(got, new, cs[60:], False)


def test_layer_trained_with_rotated_positions():
    """rope, indexer, attention and their gradients as a training step runs them, against autograd of the dense causal
    layer in 64 bits (every pool is kept at this length)."""
    S, scale = 61, 1 / math.sqrt(D)
    cs, csi = f4.table(S, 128), f4.table(S, 32)
    q, k, v, dO = bf16(S, HQ, D, seed=1), bf16(S, D, seed=2), bf16(S, D, seed=3), bf16(S, HQ, D, seed=4)
    qi, ki, w = bf16(S, 4, DI, seed=5), bf16(S, DI, seed=6), torch.rand(S, 4, generator=torch.Generator().manual_seed(7))
    rope, rope_idx = dsa.Rope(cs.to(DEV)), dsa.Rope(csi.to(DEV), interleaved=True)
    qr, kr = dsa.dsa_rope(q.to(DEV), rope), dsa.dsa_rope(k.to(DEV), rope)
    pool_idx = dsa.dsa_index_topk(dsa.dsa_rope(qi.to(DEV), rope_idx), dsa.dsa_rope(ki.to(DEV), rope_idx), w.to(DEV),
                                  chunk=16, topk=16)
    vg, dOg = v.to(DEV), dO.to(DEV)
    o, lse = dsa.dsa_sparse_attn_fwd(qr, kr, vg, pool_idx, scale=scale)
    dq, dk, dv = dsa.dsa_sparse_attn_bwd(dOg, qr, kr, vg, o, lse, pool_idx, scale=scale)
    dq, dk = dsa.dsa_rope(dq, rope, inverse=True), dsa.dsa_rope(dk, rope, inverse=True)
    dsa.dsa_sync_status()
    q2, k2, v2 = (t.double().requires_grad_() for t in (q, k, v))

    def turned(x):
        a, b = x[..., :64], x[..., 64:]
        c, s = cs[:, None, :64].double(), cs[:, None, 64:].double()
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    x = torch.einsum("ihd,jd->hij", turned(q2), turned(k2[:, None])[:, 0]) * scale
    x = x.masked_fill(torch.ones(S, S).triu(1).bool(), -math.inf)
    ro = torch.einsum("hij,jd->ihd", torch.softmax(x, -1), v2)
    ro.backward(dO.double())
    for got, ref in ((o, ro), (dq, q2.grad), (dk, k2.grad), (dv, v2.grad)):
        ref = ref.detach()
        err = (got.cpu().double() - ref).abs()
        # the layer's own tolerance, the rounding of the turned operands to bf16 (2^-8 of them) and of the gradients
        assert torch.all(err <= 2 * MAX_ABS + 2.0 ** -7 * ref.abs()) and err.norm() <= 2 * REL_L2 * ref.norm()


# --------------------------------------------------------------------------- appends

KINDS = {"whole": (128, 64, False), "pairs": (64, 32, True), "odd": (96, 48, False), "keys": (32, 0, False),
         "indexer": (0, 16, True), "none": (0, 0, False)}


def queries(m, kind, rows, seed=9):
    dims, dims_idx, _ = KINDS[kind]
    return (bf16(rows, HQ, D, seed=seed) if dims else None, bf16(rows, 6, DI, seed=seed + 1) if dims_idx else None)


def check_queries(m, ropes, given, got):
    for x, cs, y in ((given[0], ropes.k, got[0]), (given[1], ropes.idx, got[1])):
        assert (x is None) == (y is None)
        if x is not None:
            pos = torch.tensor([i for _, _, i in m.rows()])
            check_turned(y[:m.T], x[:m.T], cs[pos], ropes.inter)


def gpu(*tensors):
    return [None if t is None else t.to(DEV) for t in tensors]


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", KINDS)
def test_append_rope_bit_exact(layout, page, kind):
    """Keys as correctly rounded, pooled keys from them, everything else in the cache as it was."""
    m = f4.TurnedModel(*LAYOUTS[layout], page, seed=1)
    ropes = f4.Turned(*KINDS[kind], 200)
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    given = queries(m, kind, m.T)
    r, ri = ropes.to_gpu(dsa)
    got = dsa.dsa_cache_append_rope(cache, batch, *gpu(k, v, ki), r, ri, **dict(zip(("q", "q_idx"), gpu(*given))))
    dsa.dsa_sync_status()
    m.append_turned(ropes, k, v, ki)
    check_cache(cache, m)
    check_queries(m, ropes, given, got)


@pytest.mark.parametrize("new", [[1020, 4], [1021, 4], [700, 0, 1, 933, 2]])
@pytest.mark.parametrize("kind", ["whole", "odd", "pairs"])
def test_append_rope_of_many_rows(new, kind):
    """A warp to a row up to 1024 rows, a warp to four beyond; rows and pools that end anywhere in a warp's four."""
    m = f4.TurnedModel(new, [61, 3, 2, 0, 5][:len(new)], 32, seed=2, pages_apart=72)
    ropes = f4.Turned(*KINDS[kind], 1200, apart=4)
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    given = queries(m, kind, m.T)
    r, ri = ropes.to_gpu(dsa)
    got = dsa.dsa_cache_append_rope(cache, batch, *gpu(k, v, ki), r, ri, *gpu(*given))
    dsa.dsa_sync_status()
    m.append_turned(ropes, k, v, ki)
    check_cache(cache, m)
    check_queries(m, ropes, given, got)


@pytest.mark.parametrize("new", [[5, 40, 1], [800, 400, 3]])
def test_append_rope_of_strided_rows_with_padding(new):
    """Everything out of one fused projection, queries in place or into given outputs, rows behind the last sequence."""
    m = f4.TurnedModel(new, [2, 7, 100], 32, seed=3)
    ropes = f4.Turned(128, 64, False, 1000)
    cache, batch = m.to_gpu(dsa)
    rows, Hi = m.T + 9, 3
    widths = [HQ * D, Hi * DI, D, D, DI]
    cuts = [8]
    for n in widths:
        cuts.append(cuts[-1] + n)
    fused = bf16(rows, cuts[-1] + 8, seed=4)

    def parts(t):
        p = [t[:, a:b] for a, b in zip(cuts, cuts[1:])]
        return p[0].unflatten(1, (HQ, D)), p[1].unflatten(1, (Hi, DI)), p[2], p[3], p[4]

    q, qi, k, v, ki = parts(fused)
    t = fused.to(DEV)
    gq, gqi, gk, gv, gki = parts(t)
    r, ri = ropes.to_gpu(dsa)
    out = torch.full((rows, Hi, DI), 2.0, dtype=torch.bfloat16, device=DEV)
    a, b = dsa.dsa_cache_append_rope(cache, batch, gk, gv, gki, r, ri, q=gq, q_idx=gqi, q_out=gq, q_idx_out=out)
    dsa.dsa_sync_status()
    assert a is gq and b is out
    m.append_turned(ropes, k, v, ki)
    check_cache(cache, m)
    check_queries(m, ropes, (q, qi), (a, b))
    assert same_bits(gq[m.T:].cpu(), q[m.T:]) and torch.all(out[m.T:] == 2)
    assert same_bits(t[:, cuts[1]:].cpu(), fused[:, cuts[1]:]) and same_bits(t[:, :8].cpu(), fused[:, :8])


@pytest.mark.parametrize("new", [[4, 3, 2], [1500, 3, 2]])
def test_append_rope_of_positions_past_the_table(new):
    """Rows within the table are written, the others and their queries are not; the status says so."""
    m = f4.TurnedModel(new, [0, 30, 12], 16, seed=5)
    ropes = f4.Turned(64, 64, False, 4000)
    end = 32  # the second sequence's last row stands at 32
    cache, batch = m.to_gpu(dsa)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI)
    q = bf16(m.T, HQ, D)
    out = torch.full((m.T, HQ, D), 5.0, dtype=torch.bfloat16, device=DEV)
    r, ri = ropes.to_gpu(dsa)
    short = dsa.Rope(r.cos_sin[:end].contiguous())
    reported(lambda: dsa.dsa_cache_append_rope(cache, batch, *gpu(k, v, ki), short, ri, q=q.to(DEV), q_out=out))
    kt, it = k.clone(), ki.clone()
    for row, b, i in m.rows():
        if i < end:
            kt[row], it[row] = ropes.key(k[row], i), ropes.key_idx(ki[row], i)
            s = m.slot(b, i)
            m.k.view(-1, D)[s], m.v.view(-1, D)[s], m.k_idx.view(-1, DI)[s] = kt[row], v[row], it[row]
    for n in ("k", "v", "k_idx"):
        assert same_bits(getattr(cache, n).cpu(), getattr(m, n)), n
    pos = torch.tensor([i for _, _, i in m.rows()])
    check_turned(out[(pos < end).to(DEV)], q[pos < end], ropes.k[pos[pos < end]], False)
    assert torch.all(out[(pos >= end).to(DEV)] == 5.0)


@pytest.mark.parametrize("four", [False, True])
def test_append_rope_writes_nothing_after_a_failed_reservation_or_wrong_offsets(four):
    m = f4.Model4([3, 2], [5, 6], 16, seed=6)
    ropes = f4.Turned(64, 64, True, 100)
    cache, batch = m.to_gpu4(dsa) if four else m.to_gpu(dsa)
    call = dsa.dsa_cache4_append if four else dsa.dsa_cache_append_rope
    new = gpu(m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI))
    q = bf16(m.T, HQ, D).to(DEV)
    r, ri = ropes.to_gpu(dsa)
    out = torch.full_like(q, 5.0)
    names = ("kv", "k_idx", "khat") if four else ("k", "v", "k_idx", "khat")
    want = [getattr(cache, n).clone() for n in names]
    reported(lambda: call(cache, batch, *new, r, ri, q=q, q_out=out, reserved=i32([-2])))
    assert torch.all(out == 5.0)
    for cu in ([0, 4, 3], [0, 3, 6], [-1, 3, 5]):
        bad = dsa.PagedBatch(batch.block_table, batch.seq_lens, i32(cu))
        reported(lambda: call(cache, bad, *new, r, ri))
    for n, w in zip(names, want):
        assert torch.equal(getattr(cache, n).view(torch.int16 if n != "kv" else torch.uint8), w.view(torch.int16 if n != "kv" else torch.uint8))
    call(cache, batch, *new, r, ri, reserved=i32([0]))
    dsa.dsa_sync_status()
    m.append4(*[t.cpu() for t in new], ropes) if four else m.append_turned(ropes, *[t.cpu() for t in new])
    for n in names:
        assert torch.equal(getattr(cache, n).cpu().view(torch.uint8), getattr(m, n).view(torch.uint8)), n


@pytest.mark.parametrize("what", ["offsets", "first_offset", "middle_offsets", "reserved", "table", "table_idx", "page"])
@pytest.mark.parametrize("new", [[3, 2, 1], [1] * 290 + [3], [1500, 3, 2]])
@pytest.mark.parametrize("four", [False, True])
def test_queries_of_rows_that_are_not_appended_stay(four, new, what):
    """Turned in place: a step that is repeated after an error turns no query twice.  Offsets that are wrong anywhere, a
    failed reservation: no row is appended; a position that one of the tables does not have, a bad page: not that row."""
    m = f4.Model4(new, [2 + 7 * j % 40 for j in range(len(new))], 16, seed=12)
    ropes = f4.Turned(128, 64, False, 4000)
    cache, batch = m.to_gpu4(dsa) if four else m.to_gpu(dsa)
    call = dsa.dsa_cache4_append if four else dsa.dsa_cache_append_rope
    kvi = gpu(m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI))
    q, qi = bf16(m.T, HQ, D, seed=2), bf16(m.T, 6, DI, seed=3)
    gq, gqi = gpu(q, qi)
    r, ri = ropes.to_gpu(dsa)
    pos = torch.tensor([i for _, _, i in m.rows()])
    done, kw, br, bri, cu, table, end = torch.zeros(m.T, dtype=torch.bool), {}, r, ri, list(m.cu), m.table.clone(), 10
    if what == "offsets":
        cu[-1] += 1
    elif what == "first_offset":
        cu[0] = -1
    elif what == "middle_offsets":
        cu[-2] = cu[-1] + 1
    elif what == "reserved":
        kw = dict(reserved=i32([-1]))
    elif what == "page":
        table[1, 0] = m.pages
        done = torch.tensor([b != 1 or i >= 16 for _, b, i in m.rows()])
    else:
        done = pos < end
        br, bri = (dsa.Rope(x.cos_sin[:end].contiguous()) if (what == "table") == (x is r) else x for x in (r, ri))
    bad = dsa.PagedBatch(table.to(DEV), batch.seq_lens, i32(cu))
    reported(lambda: call(cache, bad, *kvi, br, bri, q=gq, q_idx=gqi, q_out=gq, q_idx_out=gqi, **kw))
    for given, got, cs in ((q, gq, ropes.k), (qi, gqi, ropes.idx)):
        assert same_bits(got.cpu()[~done], given[~done])
        check_turned(got[done.to(DEV)], given[done], cs[pos[done]], False)
    assert done.any() == (what in ("table", "table_idx", "page")) and not done.all()


def test_serving_with_rotated_positions_is_the_turned_training_forward():
    """A prompt in chunks, then tokens one by one, into a bf16 cache, keys, queries and indexer turned by the append:
    every row's attention is the contiguous layer's on heads that dsa_rope turned (which may round a number the other
    way: 2^-8 of it), with every pool kept."""
    S, topk, Hi = 90, 24, 4
    ropes = f4.Turned(128, 32, False, S)
    r, ri = ropes.to_gpu(dsa)
    q, k, v = bf16(S, HQ, D, seed=1).to(DEV), bf16(S, D, seed=2).to(DEV), bf16(S, D, seed=3).to(DEV)
    qi, ki = bf16(S, Hi, DI, seed=4).to(DEV), bf16(S, DI, seed=5).to(DEV)
    w = torch.rand(S, Hi, generator=torch.Generator().manual_seed(6)).to(DEV)
    cache = dsa.PagedCache.empty(8, 16)
    t = dsa.PageTable.empty(cache, max_seqs=2, max_pages=7)
    got, gl, at = [], [], 0
    for n in (33, 50, 1, 1, 1, 4):
        taken = dsa.dsa_cache_reserve(cache, t, i32([0, n]))
        batch = dsa.PagedBatch(t.block_table, t.seq_lens, i32([0, 0, n]))
        m = slice(at, at + n)
        qt, qit = dsa.dsa_cache_append_rope(cache, batch, k[m], v[m], ki[m], r, ri, q[m], qi[m], reserved=taken)
        sel = dsa.dsa_paged_index_topk(cache, batch, qit, w[m], topk)
        o, lse = dsa.dsa_paged_sparse_attn_fwd(cache, batch, qt, sel)
        got.append(o), gl.append(lse)
        at += n
    sel = dsa.dsa_index_topk(dsa.dsa_rope(qi, ri), dsa.dsa_rope(ki, ri), w, chunk=32, topk=topk)
    wo, wl = dsa.dsa_sparse_attn_fwd(dsa.dsa_rope(q, r), dsa.dsa_rope(k, r), v, sel)
    dsa.dsa_sync_status()
    torch.testing.assert_close(torch.cat(got).float(), wo.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    torch.testing.assert_close(torch.cat(gl), wl, rtol=2.0 ** -8, atol=2.0 ** -8)


def test_append_without_ropes_is_the_plain_append():
    m = f4.TurnedModel([37, 130, 5], [0, 61, 3], 64, seed=7)
    a, batch = m.to_gpu(dsa)
    b, _ = m.to_gpu(dsa)
    new = gpu(m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI))
    dsa.dsa_cache_append(a, batch, *new)
    assert dsa.dsa_cache_append_rope(b, batch, *new, None) == (None, None)
    dsa.dsa_sync_status()
    for n in ("k", "v", "k_idx", "khat"):
        assert same_bits(getattr(a, n), getattr(b, n))


def test_refusals_of_the_binding():
    m = f4.Model4([2], [30], 16, seed=8)
    cache, batch = m.to_gpu(dsa)
    cache4, _ = m.to_gpu4(dsa)
    new = gpu(m.fill(2, D), m.fill(2, D), m.fill(2, DI))
    rope = dsa.Rope(f4.table(40, 64).to(DEV))
    q = bf16(2, HQ, D).to(DEV)
    for bad in (lambda: dsa.dsa_cache_append_rope(cache4, batch, *new, rope), lambda: dsa.dsa_cache4_append(cache, batch, *new),
                lambda: dsa.dsa_cache_append(cache4, batch, *new), lambda: dsa.dsa_cache4_read(cache, batch, 2),
                lambda: dsa.dsa_paged_sparse_attn_fwd(cache4, batch, q, i32([0, 1]).view(2, 1)),
                lambda: dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q, i32([0, 1]).view(2, 1)),
                lambda: dsa.dsa_cache_copy_pages([cache, cache4], i32([0]), i32([1])),
                lambda: dsa.dsa_cache_append_rope(cache, batch, *new, f4.table(40, 64)),
                lambda: dsa.dsa_rope(q.float(), rope), lambda: dsa.dsa_rope(q, f4.table(40, 64).to(DEV)), lambda: dsa.Rope(f4.table(40, 64).to(DEV).half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dsa.dsa_cache_append_rope(cache, batch, *new, rope, q=q[:1]),
                lambda: dsa.dsa_cache_append_rope(cache, batch, *new, rope, q=q[..., :64]),
                lambda: dsa.dsa_cache_append_rope(cache, batch, *new, rope, q=q, q_out=q[:, :8]),
                lambda: dsa.dsa_cache_append_rope(cache, batch, *new, rope, q_out=q),
                lambda: dsa.dsa_cache_append_rope(cache, batch, new[0], new[1][:1], new[2], rope),
                lambda: dsa.dsa_rope(q.transpose(0, 1), rope), lambda: dsa.dsa_rope(q.cpu(), rope),
                lambda: dsa.dsa_rope(q, rope, positions=i32([1])), lambda: dsa.dsa_rope(q, rope, out=q[:1]),
                lambda: dsa.dsa_cache4_read(cache4, batch, -1),
                lambda: dsa.dsa_cache4_read(cache4, batch, 2, k=new[0][:1])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dsa.dsa_cache_append_rope(cache, batch, *new, None, q=q), lambda: dsa.dsa_rope(q, rope, q_begin=39),
                lambda: dsa.dsa_rope(bf16(2, 4, 48).to(DEV), rope), lambda: dsa.dsa_rope(q, dsa.Rope(f4.table(40, 24).to(DEV))),
                lambda: dsa.dsa_cache4_append(cache4, batch, *new, rope, dsa.Rope(f4.table(40, 128).to(DEV)))):
        with pytest.raises(dsa.DsaError) as e:
            bad()
        assert e.value.status in (dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED)


def test_calls_record_what_they_ran():
    m = f4.Model4([2], [30], 16, seed=9)
    cache, batch = m.to_gpu4(dsa)
    new = gpu(m.fill(2, D), m.fill(2, D), m.fill(2, DI))
    dsa.dsa_cache4_append(cache, batch, *new)
    c = dsa.last_kernel_config()
    assert c["entry"] == "dsa_cache4_append" and c["kernels"] == [["cache4_append", 1]]
    dsa.dsa_paged4_sparse_attn_fwd(cache, batch, bf16(2, HQ, D).to(DEV), i32([0, 1]).view(2, 1))
    c = dsa.last_kernel_config()
    assert c["entry"] == "dsa_paged4_sparse_attn_fwd" and c["kernels"] == [["paged4_attn", 1]]
    dsa.dsa_rope(bf16(2, HQ, D).to(DEV), dsa.Rope(f4.table(2, 64).to(DEV)))
    assert dsa.last_kernel_config()["kernels"] == [["rope", 1]]


def test_short_and_long_way_of_a_call_agree():
    """The extension module's way (outputs to allocate, the current stream) and the Python code's (a stream given): the
    same bits for what the first takes, and for what it leaves to the second."""
    here = torch.cuda.current_stream()
    S, wide = 20, bf16(20, 4, 256, seed=1).to(DEV)
    rope = dsa.Rope(f4.table(64, 64).to(DEV))
    pos = i32(range(3, 23))
    shapes = (wide[:, :, :128].contiguous(), wide[:, 1:2, 64:128], wide.view(20, 8, 128)[:, 2:5], wide[::2, 0, 128:],
              wide[:, 0, ::2])
    for x in shapes[:4]:
        at = pos[:x.shape[0]].contiguous()
        for kw in (dict(), dict(q_begin=9), dict(positions=at), dict(positions=at, inverse=True)):
            a, b = dsa.dsa_rope(x, rope, **kw), dsa.dsa_rope(x, rope, stream=here, **kw)
            assert same_bits(a, b) and a.shape == x.shape
    with pytest.raises(ValueError):  # a row whose elements lie apart
        dsa.dsa_rope(shapes[4], rope)
    m = f4.Model4([1, 2, 5], [7, 30, 0], 16, seed=10)
    new = gpu(m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, DI))
    q, qi = bf16(m.T, HQ, D).to(DEV), bf16(m.T, 3, DI).to(DEV)
    idx = dsa.Rope(f4.table(64, 32).to(DEV), interleaved=True)
    sel = torch.full((m.T, 4), -1, dtype=torch.int32, device=DEV)
    for four, call in ((False, dsa.dsa_cache_append_rope), (True, dsa.dsa_cache4_append)):
        for args in ((rope, idx, q, qi), (None, idx, None, qi), (rope, None, q, None), (None, None, None, None)):
            got = []
            for kw in (dict(), dict(stream=here), dict(reserved=i32([1])), dict(reserved=i32([1]), stream=here)):
                cache, batch = m.to_gpu4(dsa) if four else m.to_gpu(dsa)
                out = call(cache, batch, *new, *args, **kw)
                got.append([t for t in out if t is not None] + ([cache.kv] if four else [cache.k, cache.v])
                           + [cache.k_idx, cache.khat])
                assert [t is None for t in out] == [t is None for t in args[2:]]
                if four:
                    got[-1] += dsa.dsa_cache4_read(cache, batch, m.T, stream=kw.get("stream"))
                    got[-1] += dsa.dsa_paged4_sparse_attn_fwd(cache, batch, q, sel, 0.25, stream=kw.get("stream"))
            for other in got[1:]:
                for a, b in zip(got[0], other):
                    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    dsa.dsa_sync_status()


def test_a_direction_that_is_no_truth_value_is_refused():
    """The call's own error, whatever asking the object for its truth would raise."""
    rope, x = dsa.Rope(f4.table(8, 64).to(DEV)), bf16(8, 2, 64).to(DEV)
    for inverse in (torch.tensor([1, 2]), "back", None):
        with pytest.raises(ctypes.ArgumentError):
            dsa.dsa_rope(x, rope, inverse=inverse)
    assert same_bits(dsa.dsa_rope(x, rope, inverse=1), dsa.dsa_rope(x, rope, inverse=True))


def test_short_way_raises_what_the_library_refuses():
    rope = dsa.Rope(f4.table(8, 64).to(DEV))
    x = bf16(9, 2, 64).to(DEV)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_rope(x, rope)  # nine positions of eight
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG and "dsa_rope" in str(e.value)
    m = f4.Model4([2], [30], 16, seed=11)
    cache, batch = m.to_gpu4(dsa)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_paged4_sparse_attn_fwd(cache, batch, bf16(2, 8, 128).to(DEV), i32([0, 0]).view(2, 1))
    assert e.value.status == dsa.DSA_ERR_UNSUPPORTED
    gc.collect()
    before = torch.cuda.memory_allocated()
    for _ in range(20):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_rope(x, rope, q_begin=1)
    gc.collect()
    assert torch.cuda.memory_allocated() <= before  # the outputs of refused calls are given back


def test_both_ways_fill_new_memory_where_torch_is_told_to():
    """In torch's deterministic mode new memory is filled with NaN: what a call leaves unwritten in its outputs reads alike
    on the extension module's way and on the Python code's."""
    here = torch.cuda.current_stream()
    rope = dsa.Rope(f4.table(64, 64).to(DEV))
    m = f4.Model4([2, 1], [7, 30], 16, seed=12)
    cache, batch = m.to_gpu4(dsa)
    rows = m.T + 4  # padding behind the last sequence
    x, new = bf16(rows, HQ, D).to(DEV), gpu(bf16(rows, D), bf16(rows, D), bf16(rows, DI))
    sel = torch.full((rows, 4), -1, dtype=torch.int32, device=DEV)

    def every(**kw):
        yield dsa.dsa_cache4_append(cache, batch, *new, rope, q=x, **kw)[0]
        yield from dsa.dsa_cache4_read(cache, batch, rows, **kw)
        yield from dsa.dsa_paged4_sparse_attn_fwd(cache, batch, x, sel, **kw)

    assert not torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        for kw in (dict(), dict(stream=here)):
            for y in every(**kw):
                assert torch.isfinite(y[:m.T]).all() and torch.isnan(y[m.T:]).all()
                y.fill_(1.0)  # (what its memory holds when it is given out again)
    finally:
        torch.use_deterministic_algorithms(False)
    dsa.dsa_sync_status()
