"""Rotated positions: heads turned for the training calls, and appends that turn
keys and queries on the way (argument marshalling only, as in ``_binding`` and
``_paged``)."""
from __future__ import annotations

import ctypes

import torch

from . import _binding
from ._binding import _check, _shape, load
from ._paged import (PagedBatch, PagedCache, PagedCache4, _device_of, _full, _handle, _is_cache, _new, _on_device,
                     _rows_strided)

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class _RopeStruct(ctypes.Structure):
    _fields_ = [("cos_sin", _vp), ("positions", _i64), ("stride", _i64), ("dims", _i32), ("interleaved", _i32)]


class _QueriesStruct(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_out", _vp), ("q_stride", _i64), ("q_out_stride", _i64), ("q_idx", _vp),
                ("q_idx_out", _vp), ("q_idx_stride", _i64), ("q_idx_out_stride", _i64), ("Hq", _i32), ("Hi", _i32)]


class Rope:
    """A rotation by position: cos_sin fp32 [positions, dims] holds for every
    position the cosines of its dims/2 angles and behind them the sines.  It
    turns the first ``dims`` dimensions of a head (a multiple of 16), in pairs
    (j, j + dims/2), or (2j, 2j + 1) if interleaved.  Rows may lie any multiple
    of 4 elements apart."""

    def __init__(self, cos_sin, interleaved: bool = False):
        _on_device(cos_sin, "cos_sin", torch.float32, 2)
        self.positions, self.dims = cos_sin.shape
        if self.positions < 1 or self.dims < 1 or cos_sin.stride(1) != 1:
            raise ValueError(f"cos_sin must have contiguous rows (got shape {tuple(cos_sin.shape)}, strides "
                             f"{cos_sin.stride()})")
        self.cos_sin, self.interleaved = cos_sin, bool(interleaved)
        self.device, self.device_index = cos_sin.device, cos_sin.device.index
        self._struct = _RopeStruct(cos_sin.data_ptr(), self.positions,
                                   cos_sin.stride(0) if self.positions > 1 else self.dims, self.dims, self.interleaved)
        self._ref, self._addr = ctypes.byref(self._struct), ctypes.addressof(self._struct)


def _configure_rope(lib):
    lib.dsa_rope.argtypes = [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _i64, _vp]
    lib.dsa_cache_append_rope.argtypes = [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.dsa_cache4_append.argtypes = lib.dsa_cache_append_rope.argtypes
    lib.dsa_cache4_read.argtypes = [_vp, _vp, _vp, _i64, _vp, _i64, _vp]
    for f in (lib.dsa_rope, lib.dsa_cache_append_rope, lib.dsa_cache4_append, lib.dsa_cache4_read):
        f.restype = ctypes.c_int


def _heads_strided(t, name: str, device: int):
    """[rows, heads, D] whose rows are contiguous; returns rows, heads, D and the distance between rows, which is free."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.dim() == 3 and t.get_device() == device):
        _on_device(t, name, torch.bfloat16, 3)
    n, h, d = t.shape
    apart, head, step = t.stride()
    if n > 0 and (step != 1 or (h > 1 and head != d)):
        raise ValueError(f"{name} must have contiguous rows of heads (got shape {tuple(t.shape)}, strides "
                         f"{t.stride()})")
    return n, h, d, apart if n > 1 else h * d


def _turned_out(given, name: str, like, device: int, stream):
    """(output, its distance between rows) of heads shaped as `like`."""
    if given is None:
        given = _new(like.shape, torch.bfloat16, like.device, stream)
        return given, like.shape[1] * like.shape[2]
    apart = _heads_strided(given, name, device)[3]
    _shape(given, name, like.shape)
    return given, apart


def dsa_rope(x, rope: Rope, positions=None, q_begin: int = 0, inverse: bool = False, out=None, stream=None):
    """x [S, H, D] (or [S, D]: one head) bf16, D = 64 or 128, turned by its rows'
    positions: positions int32 [S] (a packed batch), or q_begin + r for row r (a
    shard).  Rows may lie any multiple of 8 elements apart.  inverse: turned
    back, which is the rotation's gradient (dx from dy, at the same positions).
    out may be x."""
    if not isinstance(rope, Rope):
        raise TypeError(f"rope must be a Rope (got {type(rope).__name__})")
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        back = dsa_rope(x.unsqueeze(1), rope, positions, q_begin, inverse,
                        out.unsqueeze(1) if isinstance(out, torch.Tensor) and out.dim() == 2 else out, stream)
        return out if out is not None else back.squeeze(1)
    if out is None and stream is None:
        done = (_binding.marshal or _binding.load_marshal()).rope(x, positions, rope._addr, rope.device_index, q_begin, inverse)
        if done is not None:
            return _binding.outputs(done)
    dev = _device_of(rope)
    S, H, D, apart = _heads_strided(x, "x", dev)
    at = None
    if positions is not None:
        _full(positions, "positions", torch.int32, 1, dev)
        if positions.shape[0] != S:
            _shape(positions, "positions", (S,))
        at = positions.data_ptr()
    if out is None:
        out, out_apart = _new((S, H, D), torch.bfloat16, rope.device, stream), H * D
    else:
        out, out_apart = _turned_out(out, "out", x, dev, stream)
    _check(load().dsa_rope(x.data_ptr(), apart, S, H, D, rope._ref, at, q_begin, inverse, out.data_ptr(), out_apart,
                           _handle(stream, dev)))
    return out


def dsa_cache_append_rope(cache: PagedCache, batch: PagedBatch, k, v, k_idx, rope: Rope | None, rope_idx: Rope | None = None,
                          q=None, q_idx=None, q_out=None, q_idx_out=None, reserved=None, stream=None):
    """dsa_cache_append that turns k by `rope` and k_idx by `rope_idx` on the way
    (None: not turned), each row at its position, and with them the step's
    queries: q [rows, Hq, 128] by `rope`, q_idx [rows, Hi, 64] by `rope_idx`.
    Returns (q_out, q_idx_out), None for what was not given; q_out may be q.
    Queries of rows that are not appended are not written, so that a step may be
    repeated after an error.  One launch.  reserved: as in dsa_cache_append."""
    _is_cache(cache, False)
    return _append(load().dsa_cache_append_rope, cache, batch, k, v, k_idx, rope, rope_idx, q, q_idx, q_out, q_idx_out,
                   reserved, stream)


def dsa_cache4_append(cache: PagedCache4, batch: PagedBatch, k, v, k_idx, rope: Rope | None = None,
                      rope_idx: Rope | None = None, q=None, q_idx=None, q_out=None, q_idx_out=None, reserved=None,
                      stream=None):
    """dsa_cache_append_rope into a cache in 4 bits: k (turned) and v are held as
    their codes.  Without ropes, the plain append."""
    _is_cache(cache, True)
    return _append(load().dsa_cache4_append, cache, batch, k, v, k_idx, rope, rope_idx, q, q_idx, q_out, q_idx_out,
                   reserved, stream)


def _rope_ref(r, name: str, dev: int):
    if r is None:
        return None
    if not isinstance(r, Rope):
        raise TypeError(f"{name} must be a Rope or None (got {type(r).__name__})")
    if r.device_index != dev:
        _device_of(r)
    return r._ref


def _queries(t, out, name: str, rows: int, d: int, dev: int, device, stream):
    """(output, heads, [pointers and distances]) of queries to be turned."""
    n, h, last, apart = _heads_strided(t, name, dev)
    if n != rows or last != d:
        _shape(t, name, (rows, h, d))
    if out is None:
        out, to = _new((n, h, d), torch.bfloat16, device, stream), h * d
    else:
        out, to = _turned_out(out, name + "_out", t, dev, stream)
    return out, h, (t.data_ptr(), out.data_ptr(), apart, to)


_NO_QUERIES = (None, None, 0, 0)


def _append(call, cache, batch, k, v, k_idx, rope, rope_idx, q, q_idx, q_out, q_idx_out, reserved, stream):
    if q_out is None and q_idx_out is None and stream is None:
        at = cache.device_index
        r = 0 if rope is None else rope._addr if isinstance(rope, Rope) and rope.device_index == at else None
        ri = 0 if rope_idx is None else \
            rope_idx._addr if isinstance(rope_idx, Rope) and rope_idx.device_index == at else None
        if r is not None and ri is not None and batch.device_index == at:
            done = (_binding.marshal or _binding.load_marshal()).append(cache._four, cache._addr, batch._addr, at, k,
                                                                        v, k_idx, r, ri, q, q_idx, reserved)
            if done is not None:
                return _binding.outputs(done)
    dev = _device_of(cache, batch)
    r, ri = _rope_ref(rope, "rope", dev), _rope_ref(rope_idx, "rope_idx", dev)
    ks = _rows_strided(k, "k", torch.bfloat16, 128, dev)
    vs = _rows_strided(v, "v", torch.bfloat16, 128, dev)
    kis = _rows_strided(k_idx, "k_idx", torch.bfloat16, 64, dev)
    rows = k.shape[0]
    if v.shape[0] != rows or k_idx.shape[0] != rows:
        raise ValueError(f"k, v and k_idx must have the same rows (got {rows}, {v.shape[0]} and {k_idx.shape[0]})")
    if (q is None and q_out is not None) or (q_idx is None and q_idx_out is not None):
        raise ValueError("q_out and q_idx_out need q and q_idx")
    queries = None
    if q is not None or q_idx is not None:
        hq, hi, of_q, of_qi = 0, 0, _NO_QUERIES, _NO_QUERIES
        if q is not None:
            q_out, hq, of_q = _queries(q, q_out, "q", rows, 128, dev, cache.device, stream)
        if q_idx is not None:
            q_idx_out, hi, of_qi = _queries(q_idx, q_idx_out, "q_idx", rows, 64, dev, cache.device, stream)
        queries = ctypes.byref(_QueriesStruct(*of_q, *of_qi, hq, hi))
    if reserved is not None:
        _full(reserved, "reserved", torch.int32, 1, dev)
        _shape(reserved, "reserved", (1,))
        reserved = reserved.data_ptr()
    _check(call(cache._ref, batch._with_rows(rows), k.data_ptr(), ks, v.data_ptr(), vs, k_idx.data_ptr(), kis, r, ri,
                queries, reserved, _handle(stream, dev)))
    return q_out, q_idx_out


def dsa_cache4_read(cache: PagedCache4, batch: PagedBatch, rows: int, k=None, v=None, stream=None):
    """(k, v) [rows, 128] bf16 of the batch's rows as the cache holds them,
    exactly what the codes stand for.  A batch whose cu_q counts all tokens reads
    whole sequences."""
    _is_cache(cache, True)
    if k is None and v is None and stream is None and batch.device_index == cache.device_index:
        done = (_binding.marshal or _binding.load_marshal()).read(cache._addr, batch._addr, cache.device_index, rows)
        if done is not None:
            return _binding.outputs(done)
    dev = _device_of(cache, batch)
    if rows < 0:
        raise ValueError(f"rows must be >= 0 (got {rows})")
    k, ks = _row_out(k, "k", rows, dev, cache.device, stream)
    v, vs = _row_out(v, "v", rows, dev, cache.device, stream)
    _check(load().dsa_cache4_read(cache._ref, batch._with_rows(rows), k.data_ptr(), ks, v.data_ptr(), vs,
                                  _handle(stream, dev)))
    return k, v


def _row_out(t, name: str, rows: int, dev: int, device, stream):
    if t is None:
        return _new((rows, 128), torch.bfloat16, device, stream), 128
    apart = _rows_strided(t, name, torch.bfloat16, 128, dev)
    _shape(t, name, (rows, 128))
    return t, apart
