"""Host-side checks of the paged-cache entry points, and of the plain model the GPU tests compare with (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests._paged import D, DI, HQ, Model, pool_mean, random_selection, split_hi_lo, top_pools  # noqa: E402

FAKE = 0x10000  # 16-byte aligned dummy address: the calls below fail their checks before any device access


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_index_gb300 import build as b
    b.build()
    import long_context_sparse_index_gb300 as dsa
    return dsa.load()


def structs(**kw):
    from long_context_sparse_index_gb300 import _paged as p
    a = dict(k=FAKE, v=FAKE, k_idx=FAKE, khat=FAKE, ks=2048, vs=2048, kis=1024, khs=512, num_pages=10, page=16, D=128,
             Di=64, table=FAKE, stride=8, lens=FAKE, cu=FAKE, rows=4, max_pages=8, batch=2, count=FAKE, max_seqs=2,
             t_pages=10, t_page=16)
    assert set(kw) <= set(a)
    a.update(kw)
    c = p._CacheStruct(a["k"], a["v"], a["k_idx"], a["khat"], a["ks"], a["vs"], a["kis"], a["khs"], a["num_pages"],
                       a["page"], a["D"], a["Di"])
    b = p._BatchStruct(a["table"], a["stride"], a["lens"], a["cu"], a["rows"], a["max_pages"], a["batch"])
    t = p._TableStruct(a["table"], a["stride"], a["lens"], a["count"], a["t_pages"], a["max_pages"], a["max_seqs"],
                       a["t_page"])
    return ctypes.byref(c), ctypes.byref(b), ctypes.byref(t)


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 30


def index(lib, q=FAKE, w=FAKE, Hi=4, Di=64, topk=8, out=FAKE, ws=FAKE, size=BIG, **kw):
    c, b, _ = structs(**kw)
    return lib.dsa_paged_index_topk(c, b, q, w, Hi, Di, topk, out, ws, size, None)


def attn(lib, q=FAKE, sel=FAKE, Hq=16, D=128, topk=8, o=FAKE, lse=FAKE, scale=0.0, **kw):
    c, b, _ = structs(**kw)
    return lib.dsa_paged_sparse_attn_fwd(c, b, q, sel, Hq, D, topk, scale, o, lse, None)


def append(lib, nk=FAKE, nv=FAKE, nki=FAKE, sk=128, sv=128, ski=64, **kw):
    c, b, _ = structs(**kw)
    return lib.dsa_cache_append(c, b, nk, sk, nv, sv, nki, ski, None)


@pytest.mark.parametrize("call", [index, attn, append])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(khat=None), INVALID), (dict(k_idx=FAKE + 8), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(Di=128), UNSUPPORTED),
    (dict(ks=2047), INVALID), (dict(vs=2052), INVALID), (dict(kis=1016), INVALID),
    (dict(khs=504), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 28), INVALID), (dict(table=None), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(cu=None), INVALID), (dict(batch=0), INVALID), (dict(batch=8193), UNSUPPORTED),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 28, stride=1 << 28), INVALID), (dict(stride=7), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 28), INVALID)])
def test_cache_and_batch_are_checked(lib, call, kw, status):
    if call is index and "Di" in kw or call is attn and "D" in kw:
        c = dict(kw)
        name = "Di" if call is index else "D"
        v = c.pop(name)
        assert call(lib, **{name: v}, **c) == status  # the call's own dimension
        return
    assert call(lib, **kw) == status
    assert lib.dsa_last_error()


def test_index_arguments_are_checked(lib):
    for kw in (dict(q=None), dict(w=None), dict(out=None), dict(q=FAKE + 8), dict(w=FAKE + 1), dict(topk=0), dict(Hi=0)):
        assert index(lib, **kw) == INVALID, kw
    assert index(lib, Hi=65) == UNSUPPORTED and index(lib, topk=2049) == UNSUPPORTED
    # 8 pages of 4 pools, 4 bytes and an eighth, 4 rows
    assert index(lib, ws=None) == WORKSPACE and index(lib, size=4 * 36 * 4 - 1) == WORKSPACE
    assert index(lib, ws=FAKE + 16) == INVALID
    assert index(lib, rows=0, q=None, w=None, out=None, ws=None, size=0) == OK  # nothing to do


def test_attention_arguments_are_checked(lib):
    for kw in (dict(q=None), dict(sel=None), dict(o=None), dict(lse=None), dict(q=FAKE + 8), dict(o=FAKE + 2),
               dict(sel=FAKE + 2), dict(lse=FAKE + 1), dict(topk=0)):
        assert attn(lib, **kw) == INVALID, kw
    assert attn(lib, Hq=8) == UNSUPPORTED and attn(lib, D=64) == UNSUPPORTED and attn(lib, topk=2049) == UNSUPPORTED
    assert attn(lib, rows=0, q=None, sel=None, o=None, lse=None) == OK


def test_append_arguments_are_checked(lib):
    for kw in (dict(nk=None), dict(nv=None), dict(nki=None), dict(nk=FAKE + 8), dict(sk=120), dict(sv=132), dict(ski=56)):
        assert append(lib, **kw) == INVALID, kw
    assert append(lib, rows=0, nk=None, nv=None, nki=None) == OK


def test_append_after_a_reservation_is_checked(lib):
    def call(reserved, rows=4, **kw):
        c, b, _ = structs(rows=rows, **kw)
        return lib.dsa_cache_append_reserved(c, b, FAKE, 128, FAKE, 128, FAKE, 64, reserved, None)
    assert call(FAKE + 2) == INVALID and b"dsa_cache_append_reserved: reserved" in lib.dsa_last_error()
    assert call(FAKE, page=24) == UNSUPPORTED and call(None, k=None) == INVALID
    assert call(FAKE, rows=0) == OK


def test_page_operators_are_checked(lib):
    c, _, t = structs()
    size = lib.dsa_cache_workspace(10, 2, 2)
    assert lib.dsa_cache_reserve(t, FAKE, FAKE, FAKE, 4, None) == WORKSPACE
    assert lib.dsa_cache_reserve(t, None, FAKE, FAKE, size, None) == INVALID
    assert lib.dsa_cache_reserve(t, FAKE, FAKE, FAKE + 4, size, None) == INVALID
    assert lib.dsa_cache_fork(c, 1, t, FAKE, FAKE, 3, FAKE, FAKE, size, None) == INVALID  # more children than rows
    assert lib.dsa_cache_fork(c, 1, t, FAKE, None, 2, FAKE, FAKE, size, None) == INVALID
    assert lib.dsa_cache_fork(c, 1, t, FAKE, FAKE, 2, FAKE, None, 0, None) == WORKSPACE
    assert lib.dsa_cache_free(t, None, 2, None) == INVALID and lib.dsa_cache_free(t, FAKE, -1, None) == INVALID
    assert lib.dsa_cache_free(t, None, 0, None) == OK
    assert lib.dsa_cache_compact(c, 1, t, None, FAKE, size, None) == INVALID
    assert lib.dsa_cache_compact(c, 1, t, FAKE, FAKE, 16, None) == WORKSPACE
    assert lib.dsa_cache_copy_pages(c, 1, None, FAKE, 1, None) == INVALID
    assert lib.dsa_cache_copy_pages(c, 1, None, None, 0, None) == OK
    for kw in (dict(t_pages=11), dict(t_page=32)):  # another cache's table
        c, _, t = structs(**kw)
        assert lib.dsa_cache_fork(c, 1, t, FAKE, FAKE, 1, FAKE, FAKE, BIG, None) == INVALID
        assert lib.dsa_cache_compact(c, 1, t, FAKE, FAKE, BIG, None) == INVALID
    for kw, status in ((dict(t_page=20), UNSUPPORTED), (dict(max_seqs=0), INVALID), (dict(count=None), INVALID),
                       (dict(stride=7), INVALID), (dict(t_pages=0), INVALID)):
        _, _, t = structs(**kw)
        assert lib.dsa_cache_free(t, FAKE, 1, None) == status, kw
        assert lib.dsa_cache_reserve(t, FAKE, FAKE, FAKE, BIG, None) == status, kw


def test_tables_of_more_rows_than_the_kernels_count_are_refused(lib):
    """The planners walk the sequences in 32-bit steps of a block or more: 2^31 - 1 rows would pass the end."""
    size = lib.dsa_cache_workspace(10, 2, 2)
    for seqs in (0, -1, (1 << 27) + 1, 2 ** 31 - 1):
        c, _, t = structs(max_seqs=seqs)
        assert lib.dsa_cache_reserve(t, FAKE, FAKE, FAKE, 1 << 40, None) == INVALID, seqs
        assert lib.dsa_cache_free(t, FAKE, 1, None) == INVALID, seqs
        assert lib.dsa_cache_fork(c, 1, t, FAKE, FAKE, 1, FAKE, FAKE, 1 << 40, None) == INVALID, seqs
        assert lib.dsa_cache_compact(c, 1, t, FAKE, FAKE, size, None) == INVALID, seqs
        assert lib.dsa_cache_workspace(10, seqs, 0) == 0
    assert lib.dsa_cache_workspace(10, 1 << 27, 0) == ((1 << 27) + 10) * 4 // 256 * 256 + 256


def test_layers_are_checked(lib):
    from long_context_sparse_index_gb300 import _paged as p
    one, _, t = structs()
    size = lib.dsa_cache_workspace(10, 2, 2)
    assert lib.dsa_cache_copy_pages(one, 0, FAKE, FAKE, 1, None) == INVALID
    assert lib.dsa_cache_copy_pages(None, 1, FAKE, FAKE, 1, None) == INVALID
    a = structs()[0]._obj
    for kw in (dict(num_pages=11), dict(page=32, ks=4096, vs=4096, kis=2048, khs=1024), dict(v=None)):
        two = (p._CacheStruct * 2)(a, structs(**kw)[0]._obj)
        assert lib.dsa_cache_copy_pages(two, 2, FAKE, FAKE, 1, None) == INVALID, kw
        assert lib.dsa_cache_fork(two, 2, t, FAKE, FAKE, 1, FAKE, FAKE, size, None) == INVALID, kw
        assert lib.dsa_cache_compact(two, 2, t, FAKE, FAKE, size, None) == INVALID, kw


def test_workspace_sizes(lib):
    r = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert lib.dsa_cache_workspace(1000, 8, 0) == r((4 + 3 * 1000) * 4)
    assert lib.dsa_cache_workspace(10, 500, 400) == r((4 + 1200 + 500) * 4)
    assert lib.dsa_cache_workspace(0, 8, 0) == 0 and lib.dsa_cache_workspace(10, 0, 0) == 0
    assert lib.dsa_paged_index_topk_workspace(64, 2050, 64) == 64 * 2050 * 18 * 4
    assert lib.dsa_paged_index_topk_workspace(3, 5, 16) == r(3 * 36 * 4)
    # a pass stays under 1 GiB, and takes at least 8 rows
    assert lib.dsa_paged_index_topk_workspace(100000, 2050, 64) <= (1 << 30) * 9 // 8
    assert lib.dsa_paged_index_topk_workspace(100, 1 << 20, 1024) == 8 * (1 << 28) * 9 // 2
    assert lib.dsa_paged_index_topk_workspace(0, 5, 16) == 0 and lib.dsa_paged_index_topk_workspace(3, 5, 24) == 0


# --------------------------------------------------------------------------- the plain model against the oracle

def test_model_agrees_with_the_oracle():
    """The paged model's pooling, selection and attention are the layer's: the same numbers as the oracle's on one
    contiguous sequence."""
    import oracle
    m = Model([45], [0], 16, seed=5, ints=True)
    k, v, ki = m.fill(45, D), m.fill(45, D), m.fill(45, DI)
    m.append(k, v, ki)
    g = torch.Generator().manual_seed(6)
    q = torch.randint(-3, 4, (45, 3, DI), generator=g).to(torch.bfloat16)
    w = torch.randint(0, 4, (45, 3), generator=g).float()
    bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    ref, _ = oracle.index_topk(bits(q), bits(ki), w.numpy(), 6)
    scores, _ = m.scores(q, w)
    assert np.array_equal(np.stack([top_pools(s, 6) for s in scores]), ref)
    qa = torch.randn(45, HQ, D, generator=g).to(torch.bfloat16)
    o, lse, _, _ = m.attention(qa, torch.from_numpy(ref), 0.1)
    ro, rl = oracle.attn_fwd(bits(qa), bits(k), bits(v), ref, scale=0.1)
    np.testing.assert_allclose(o.numpy(), ro, rtol=1e-10, atol=1e-10)
    np.testing.assert_allclose(lse.numpy(), rl, rtol=1e-10, atol=1e-10)


def test_model_selection_is_valid():
    m = Model([3, 1], [20, 0], 16, seed=1)
    sel = random_selection(m, 4, seed=2).numpy()
    for r, _, i in m.rows():
        n = min(4, i // 4)
        assert np.all(sel[r, n:] == -1) and np.all(np.diff(sel[r, :n]) > 0) and np.all(sel[r, :n] < max(i // 4, 1))
