"""Host-side checks of the rotated and 4-bit entry points, and of the plain models the GPU tests compare with (no GPU)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
from tests import _four as f4  # noqa: E402
from tests._paged import D, Model  # noqa: E402
from tests.test_paged_cpu import BIG, FAKE, INVALID, OK, UNSUPPORTED, WORKSPACE, structs  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_index_gb300 import build as b
    b.build()
    import long_context_sparse_index_gb300 as dsa
    return dsa.load()


def rope_struct(cs=FAKE, positions=100, stride=64, dims=64, inter=0):
    from long_context_sparse_index_gb300 import _rope as r
    return ctypes.byref(r._RopeStruct(cs, positions, stride, dims, inter))


def cache4(kv=FAKE, k_idx=FAKE, khat=FAKE, kvs=2304, kis=1024, khs=512, num_pages=10, page=16, D=128, Di=64):
    from long_context_sparse_index_gb300 import _paged as p
    return ctypes.byref(p._Cache4Struct(kv, k_idx, khat, kvs, kis, khs, num_pages, page, D, Di))


def queries(**kw):
    from long_context_sparse_index_gb300 import _rope as r
    a = dict(q=FAKE, q_out=FAKE, q_stride=2048, q_out_stride=2048, q_idx=FAKE, q_idx_out=FAKE, q_idx_stride=512,
             q_idx_out_stride=512, Hq=16, Hi=8)
    assert set(kw) <= set(a)
    a.update(kw)
    return ctypes.byref(r._QueriesStruct(**a))


def rope(lib, x=FAKE, xs=1024, rows=4, heads=16, D=64, r=None, positions=None, begin=0, inverse=0, out=FAKE, os=1024):
    return lib.dsa_rope(x, xs, rows, heads, D, rope_struct() if r is None else r, positions, begin, inverse, out, os, None)


def append(lib, four, r="", ri="", q=None, reserved=None, c4=None, nk=FAKE, nv=FAKE, nki=FAKE, sk=128, sv=128, ski=64, **kw):
    c, b, _ = structs(**kw)
    r = rope_struct(dims=128, stride=128) if r == "" else r
    ri = rope_struct() if ri == "" else ri
    if four:
        return lib.dsa_cache4_append(c4 or cache4(), b, nk, sk, nv, sv, nki, ski, r, ri, q, reserved, None)
    return lib.dsa_cache_append_rope(c, b, nk, sk, nv, sv, nki, ski, r, ri, q, reserved, None)


def test_rope_arguments_are_checked(lib):
    for kw, status in (
            (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID),
            (dict(xs=1016), INVALID), (dict(xs=1028), INVALID), (dict(os=1020), INVALID), (dict(os=2048), INVALID),
            (dict(heads=0), INVALID), (dict(heads=-1), INVALID), (dict(heads=129, xs=129 * 64, os=129 * 64), UNSUPPORTED),
            (dict(D=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID),
            (dict(begin=-1), INVALID), (dict(begin=97), INVALID), (dict(begin=2 ** 63 - 1), INVALID),
            (dict(positions=FAKE + 2), INVALID),
            (dict(r=rope_struct(cs=None)), INVALID), (dict(r=rope_struct(cs=FAKE + 8)), INVALID),
            (dict(r=rope_struct(positions=0)), INVALID), (dict(r=rope_struct(positions=1 << 31)), INVALID),
            (dict(r=rope_struct(stride=60)), INVALID), (dict(r=rope_struct(stride=66)), INVALID),
            (dict(r=rope_struct(dims=0)), UNSUPPORTED), (dict(r=rope_struct(dims=24)), UNSUPPORTED),
            (dict(r=rope_struct(dims=128, stride=128)), UNSUPPORTED), (dict(r=rope_struct(dims=-16)), UNSUPPORTED)):
        assert rope(lib, **kw) == status, kw
        assert lib.dsa_last_error()
    assert lib.dsa_rope(FAKE, 1024, 4, 16, 64, None, None, 0, 0, FAKE, 1024, None) == INVALID
    assert rope(lib, rows=0, x=None, out=None) == OK
    assert rope(lib, rows=0, begin=100) == OK and rope(lib, rows=0, begin=101) == INVALID


@pytest.mark.parametrize("four", [False, True])
def test_append_arguments_are_checked(lib, four):
    for kw in (dict(nk=None), dict(nv=None), dict(nki=None), dict(nk=FAKE + 8), dict(sk=120), dict(sv=132),
               dict(ski=56), dict(reserved=FAKE + 2), dict(batch=0), dict(rows=-1), dict(table=None),
               dict(r=rope_struct(cs=None, dims=128, stride=128)), dict(ri=rope_struct(cs=FAKE + 4)),
               dict(r=None, q=queries()), dict(ri=None, q=queries()), dict(q=queries(q=None)),
               dict(q=queries(q_out=FAKE + 8)), dict(q=queries(q_stride=2040)), dict(q=queries(q_idx_stride=516)),
               dict(q=queries(q_idx_out=None)), dict(q=queries(q_out_stride=4096))):  # (in place with another stride)
        assert append(lib, four, **kw) == INVALID, kw
    for kw in (dict(r=rope_struct(dims=144, stride=144)), dict(ri=rope_struct(dims=80, stride=80)),
               dict(q=queries(Hq=129)), dict(q=queries(Hi=65)), dict(q=queries(Hq=-1)), dict(batch=8193)):
        assert append(lib, four, **kw) == UNSUPPORTED, kw
    name = b"dsa_cache4_append" if four else b"dsa_cache_append_rope"
    append(lib, four, nk=None)
    assert name in lib.dsa_last_error()
    assert append(lib, four, rows=0, nk=None, nv=None, nki=None, q=queries(q=None)) == OK
    assert append(lib, four, rows=0, r=None, q=queries(Hi=0)) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(kv=None), INVALID), (dict(k_idx=None), INVALID), (dict(khat=None), INVALID), (dict(kv=FAKE + 8), INVALID),
    (dict(kvs=2303), INVALID), (dict(kvs=2288), INVALID), (dict(kvs=2312), INVALID), (dict(kis=1016), INVALID),
    (dict(khs=516), INVALID), (dict(num_pages=0), INVALID), (dict(num_pages=1 << 28), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(Di=128), UNSUPPORTED)])
def test_caches_in_4_bits_are_checked(lib, kw, status):
    c = cache4(**kw)
    _, b, t = structs(**({"page": 16} if "page" not in kw else {}))
    assert append(lib, True, c4=c) == status
    assert lib.dsa_cache4_read(c, b, FAKE, 128, FAKE, 128, None) == status
    assert lib.dsa_cache4_copy_pages(c, 1, FAKE, FAKE, 1, None) == status
    assert lib.dsa_cache4_fork(c, 1, t, FAKE, FAKE, 1, FAKE, FAKE, BIG, None) == status
    assert lib.dsa_cache4_compact(c, 1, t, FAKE, FAKE, BIG, None) == status
    assert lib.dsa_paged4_index_topk(c, b, FAKE, FAKE, 4, 64, 8, FAKE, FAKE, BIG, None) == status
    assert lib.dsa_paged4_sparse_attn_fwd(c, b, FAKE, FAKE, 16, 128, 8, 0.0, FAKE, FAKE, None) == status
    assert lib.dsa_last_error()


def test_calls_over_4_bits_check_their_arguments(lib):
    c, (_, b, t) = cache4(), structs()
    for args in ((None, 128, FAKE, 128), (FAKE, 128, None, 128), (FAKE + 8, 128, FAKE, 128), (FAKE, 120, FAKE, 128),
                 (FAKE, 128, FAKE, 132)):
        assert lib.dsa_cache4_read(c, b, *args, None) == INVALID, args
    assert lib.dsa_cache4_read(c, structs(rows=0)[1], None, 0, None, 0, None) == OK
    assert lib.dsa_cache4_read(c, None, FAKE, 128, FAKE, 128, None) == INVALID
    assert lib.dsa_paged4_sparse_attn_fwd(c, b, FAKE, FAKE, 8, 128, 8, 0.0, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.dsa_paged4_sparse_attn_fwd(c, b, FAKE, FAKE, 16, 128, 2049, 0.0, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.dsa_paged4_sparse_attn_fwd(c, b, FAKE, FAKE, 16, 128, 0, 0.0, FAKE, FAKE, None) == INVALID
    assert lib.dsa_paged4_sparse_attn_fwd(c, b, FAKE + 8, FAKE, 16, 128, 8, 0.0, FAKE, FAKE, None) == INVALID
    assert lib.dsa_paged4_index_topk(c, b, FAKE, FAKE, 65, 64, 8, FAKE, FAKE, BIG, None) == UNSUPPORTED
    assert lib.dsa_paged4_index_topk(c, b, FAKE, FAKE, 4, 64, 8, FAKE, None, 0, None) == WORKSPACE
    assert lib.dsa_cache4_copy_pages(c, 0, FAKE, FAKE, 1, None) == INVALID
    assert lib.dsa_cache4_copy_pages(c, 1, FAKE, None, 1, None) == INVALID
    assert lib.dsa_cache4_copy_pages(c, 1, None, None, 0, None) == OK
    for kw in (dict(t_pages=11), dict(t_page=32)):  # another cache's table
        other = structs(**kw)[2]
        assert lib.dsa_cache4_fork(c, 1, other, FAKE, FAKE, 1, FAKE, FAKE, BIG, None) == INVALID
        assert lib.dsa_cache4_compact(c, 1, other, FAKE, FAKE, BIG, None) == INVALID
    from long_context_sparse_index_gb300 import _paged as p
    two = (p._Cache4Struct * 2)(cache4()._obj, cache4(num_pages=11)._obj)  # layers whose pages differ
    assert lib.dsa_cache4_copy_pages(two, 2, FAKE, FAKE, 1, None) == INVALID


def test_binding_refuses_what_is_no_rope_and_cpu_tensors():
    import long_context_sparse_index_gb300 as dsa
    with pytest.raises(ValueError):
        dsa.Rope(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        dsa.dsa_cache4_append(object(), None, None, None, None)
    with pytest.raises(TypeError):
        dsa.dsa_paged4_sparse_attn_fwd(None, None, None, None)


def test_library_loads_without_a_fitting_extension_module(lib, monkeypatch):
    """A module that is missing, or of another torch: a warning, and every call is left to the Python code."""
    import sys
    import types

    from long_context_sparse_index_gb300 import _binding
    monkeypatch.setattr(_binding, "marshal", None)
    pkg = sys.modules["long_context_sparse_index_gb300"]
    for module in (None, types.SimpleNamespace(torch_version="0.0", bind=lambda *a: pytest.fail("bound"))):
        monkeypatch.setitem(sys.modules, "long_context_sparse_index_gb300._marshal", module)
        if module is None:
            monkeypatch.delattr(pkg, "_marshal", raising=False)
        else:
            monkeypatch.setattr(pkg, "_marshal", module, raising=False)
        with pytest.warns(RuntimeWarning, match="_marshal.so"):
            _binding._bind_marshal(lib)
        m = _binding.load_marshal()
        assert [f() for f in (m.rope, m.append, m.read, m.attention4)] == [None] * 4


# --------------------------------------------------------------------------- the plain models

def test_scales_and_codes_are_exact_in_16_bits():
    """Every value that the format holds is an fp16 number (times 16) and a bf16 number."""
    every = (SCALES := f4.SCALES)[:, None] * f4.SIZES
    assert torch.equal(every.half().double(), every) and every.max() == 61440
    assert torch.equal((every / 16).to(torch.bfloat16).double(), every / 16)
    assert torch.equal((torch.arange(0xE3, dtype=torch.int16) << 7).view(torch.float16).double(), SCALES)


def test_quantiser_agrees_with_the_formula():
    """Nearest of all numbers, by rounding to the number of digits that the format has there."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(400, 128, generator=g, dtype=torch.float64) *
         2.0 ** torch.randint(-30, 14, (400, 1), generator=g)).to(torch.bfloat16)
    code, bits = f4.quantise(x)
    y = 16 * x.double().view(-1, 8, 16)
    m = (y.abs().amax(2) / 6).clamp(min=1e-30)
    e = torch.floor(torch.log2(m)).clamp(min=-14)
    s = (torch.round(m / 2 ** (e - 3)) * 2 ** (e - 3)).clamp(max=10240)
    assert torch.equal(f4.SCALES[bits], s)
    r = torch.where(s[..., None] > 0, y.abs() / s[..., None], 0.0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    want = (torch.round(r / step) * step).clamp(max=6) * s[..., None] / 16
    assert torch.equal(f4.stands_for(code, bits).abs().view(-1, 8, 16), want)
    # within half a step of the code, and half a step of the scale's rounding (saturation at 6 of a scale rounded down)
    ok = (m < 10240) & (m > 2.0 ** -14)
    err = (want - x.double().abs().view(-1, 8, 16)).abs()
    assert (err <= (s / 16)[..., None] * (1 + 6 / 16))[ok].all()


def test_bytes_of_a_pool_come_back():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2, 4, 128, generator=g).to(torch.bfloat16)
    pool = torch.zeros(576, dtype=torch.uint8)
    q = [f4.quantise(x[h]) for h in range(2)]
    for t in range(4):
        f4.write(pool, t, (q[0][0][t], q[0][1][t]), (q[1][0][t], q[1][1][t]))
    k, v = f4.read(pool)
    assert torch.equal(k, f4.stands_for(*q[0])) and torch.equal(v, f4.stands_for(*q[1]))
    every = torch.cat([torch.cat(f4.places(t)) for t in range(4)])
    assert sorted(every.tolist()) == list(range(576))  # every byte is one token's


@pytest.mark.parametrize("inter", [False, True])
def test_turning_is_a_product_with_complex_numbers(inter):
    cs = f4.table(5, 32)
    x = torch.randn(5, 3, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    y, _ = f4.turn(x, cs, inter)
    a, b = f4.pairs(32, inter)
    z = torch.complex(x[..., a].double(), x[..., b].double()) * torch.complex(cs[:, None, :16].double(), cs[:, None, 16:].double())
    torch.testing.assert_close(torch.complex(y[..., a], y[..., b]), z, rtol=1e-12, atol=1e-12)
    assert torch.equal(y[..., 32:], x[..., 32:].double())
    back, _ = f4.turn(y, cs, inter, inverse=True)
    torch.testing.assert_close(back, x.double(), rtol=1e-6, atol=1e-6)  # the table's fp32 cosines


@pytest.mark.parametrize("inter", [False, True])
def test_turning_back_is_the_gradient(inter):
    """Against differences of the forward formula, which is linear: they are exact up to 64-bit rounding."""
    cs = f4.table(3, 16) * 1.5  # a table that is not of unit length: the gradient is the transpose, not the inverse
    g = torch.Generator().manual_seed(6)
    x, dy = torch.randn(3, 2, 64, generator=g).double(), torch.randn(3, 2, 64, generator=g).double()
    dx, _ = f4.turn(dy, cs, inter, inverse=True)
    for at in ((0, 0, 0), (1, 1, 7), (2, 0, 8), (2, 1, 15), (1, 0, 40)):
        h = torch.zeros_like(x)
        h[at] = 1e-3
        num = ((f4.turn(x + h, cs, inter)[0] - f4.turn(x - h, cs, inter)[0]) * dy).sum() / 2e-3
        assert abs(num - dx[at]) <= 1e-9 * (1 + abs(dx[at]))


def test_model_in_4_bits_holds_what_its_bytes_say():
    m = f4.Model4([5, 2], [2, 9], 16, seed=7)
    ropes = f4.Turned(64, 32, False, 20)
    k, v, ki = m.fill(m.T, D), m.fill(m.T, D), m.fill(m.T, 64)
    m.append4(k, v, ki, ropes)
    for p in range(m.pages * 4):
        kk, vv = f4.read(m.kv.view(-1, 576)[p])
        assert torch.equal(kk, m.k.view(-1, 4, D)[p].double()) and torch.equal(vv, m.v.view(-1, 4, D)[p].double())
    # positions: the second sequence's rows stand at 9 and 10
    want = f4.quantise(f4.turned_key(k[5:], ropes.k[9:11], False))
    assert torch.equal(m.k.view(-1, D)[[m.slot(1, 9), m.slot(1, 10)]].double(), f4.stands_for(*want))


def test_a_group_with_an_infinity_stands_for_nan():
    x = torch.ones(1, 128).to(torch.bfloat16)
    x[0, 20], x[0, 120] = math.inf, math.nan
    y = f4.stands_for(*f4.quantise(x))
    assert torch.isnan(y[0, 16:32]).all() and torch.isnan(y[0, 112:]).all() and torch.isfinite(y[0, 32:112]).all()


def test_plain_cache_is_the_base_models():
    """A model without ropes appends what the base model appends."""
    a, b = Model([3], [2], 16, seed=8), f4.TurnedModel([3], [2], 16, seed=8)
    k, v, ki = a.fill(3, D), a.fill(3, D), a.fill(3, 64)
    a.append(k, v, ki)
    b.append_turned(f4.Turned(0, 0, False, 10), k, v, ki)
    for n in ("k", "v", "k_idx", "khat"):
        assert torch.equal(getattr(a, n), getattr(b, n))
