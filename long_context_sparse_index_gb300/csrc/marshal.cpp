// marshal.cpp -- the Python binding's short way into the C ABI for the calls of a
// decoding step, which are bound by the host: an extension module that checks the
// tensors, allocates the outputs and calls libdsa, without the interpreter in
// between.
//
// It takes only what needs no second look: plain tensors of the expected type,
// device and layout, on the current stream, with outputs to be allocated.
// Whatever else it is given it declines (it returns None), and the Python code
// beside it does the call, or says what is wrong.  A nonzero status of the C call
// is returned as a number.
//
// Measured on the GPU's host, from Python, kernels not waited for: attention of one
// row 12.9 -> 4.6 us, an append with queries 17.0 -> 5.6, dsa_rope 10.8 -> 4.0, of
// which the C call is 3.2 (two allocations by torch.empty take 5.7).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>

#include "../../include/dsa.h"

namespace {

using RopeFn = decltype(&dsa_rope);
using AppendFn = decltype(&dsa_cache_append_rope);
using Append4Fn = decltype(&dsa_cache4_append);
using ReadFn = decltype(&dsa_cache4_read);
using AttnFn = decltype(&dsa_paged4_sparse_attn_fwd);
struct {
  RopeFn rope;
  AppendFn append;
  Append4Fn append4;
  ReadFn read;
  AttnFn attn;
} g_lib;

PyObject* declined() { Py_RETURN_NONE; }

// A plain tensor on `device` with elements of `type` and `dims` dimensions.
const at::Tensor* plain(PyObject* o, c10::ScalarType type, int64_t dims, int device) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != device ||
      t.scalar_type() != type || t.dim() != dims)
    return nullptr;
  return &t;
}
// [rows, d] with contiguous rows; *apart: the distance between them.
const at::Tensor* rows_of(PyObject* o, int64_t d, int device, int64_t* apart) {
  const at::Tensor* t = plain(o, at::kBFloat16, 2, device);
  if (!t || t->size(1) != d || t->size(0) < 1 || t->stride(1) != 1) return nullptr;
  *apart = t->size(0) > 1 ? t->stride(0) : d;
  return t;
}
// [rows, heads, d] whose rows are contiguous.
const at::Tensor* heads_of(PyObject* o, int device, int64_t* apart) {
  const at::Tensor* t = plain(o, at::kBFloat16, 3, device);
  if (!t || t->size(0) < 1 || t->size(1) < 1 || t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != t->size(2)))
    return nullptr;
  *apart = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
  return t;
}
at::Tensor fresh(at::IntArrayRef shape, c10::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                std::nullopt);
}

// Whether the handles are on the current device, and new memory is left as it is
// (torch's deterministic mode has it filled, which torch.empty does and fresh() does
// not).
bool takes(long device) {
  at::Context& c = at::globalContext();
  if (c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory()) return false;
  return device >= 0 && c10::cuda::current_device() == device;
}
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

template <typename T>
const T* address(PyObject* o) {
  return static_cast<const T*>(PyLong_AsVoidPtr(o));
}

// C++ exceptions (out of memory among them) become Python's, as torch's own calls
// make them.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (kind) PyErr_SetString(kind, e.what_without_backtrace());
    Py_XDECREF(kind);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rope(x, positions | None, rope, device, q_begin, inverse)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const long device = n == 6 ? PyLong_AsLong(a[3]) : -1;
    const long long begin = n == 6 ? PyLong_AsLongLong(a[4]) : 0;
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return declined();
    }
    int64_t apart = 0;
    if (!takes(device) || !PyBool_Check(a[5])) return declined();
    const int d = static_cast<int>(device);
    const at::Tensor* x = heads_of(a[0], d, &apart);
    const at::Tensor* at = nullptr;
    if (!x) return declined();
    const int64_t rows = x->size(0), heads = x->size(1), dim = x->size(2);
    if (a[1] != Py_None) {
      at = plain(a[1], at::kInt, 1, d);
      if (!at || at->size(0) != rows || !at->is_contiguous()) return declined();
    }
    if (heads > 128 || dim > 256) return declined();
    at::Tensor out = fresh({rows, heads, dim}, at::kBFloat16, d);
    const dsa_rope_t* r = address<dsa_rope_t>(a[2]);
    void* stream = stream_of(d);
    const int back = a[5] == Py_True;
    dsa_status_t st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_lib.rope(x->const_data_ptr(), apart, rows, static_cast<int>(heads), static_cast<int>(dim), r,
                    at ? static_cast<const int32_t*>(at->const_data_ptr()) : nullptr, begin, back, out.mutable_data_ptr(),
                    heads * dim, stream);
    Py_END_ALLOW_THREADS;
    if (st != DSA_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(out));
  });
}

// append(four, cache, batch, device, k, v, k_idx, rope, rope_idx, q | None, q_idx | None, reserved | None):
// (q_out, q_idx_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const long device = n == 12 ? PyLong_AsLong(a[3]) : -1;
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return declined();
    }
    if (!takes(device)) return declined();
    const int d = static_cast<int>(device);
    int64_t ks = 0, vs = 0, is = 0, qs = 0, qis = 0;
    const at::Tensor *k = rows_of(a[4], 128, d, &ks), *v = rows_of(a[5], 128, d, &vs), *ki = rows_of(a[6], 64, d, &is);
    if (!k || !v || !ki || v->size(0) != k->size(0) || ki->size(0) != k->size(0)) return declined();
    const int64_t rows = k->size(0);
    const at::Tensor *q = nullptr, *qi = nullptr;
    if (a[9] != Py_None) {
      q = heads_of(a[9], d, &qs);
      if (!q || q->size(0) != rows || q->size(1) > 128 || q->size(2) != 128) return declined();
    }
    if (a[10] != Py_None) {
      qi = heads_of(a[10], d, &qis);
      if (!qi || qi->size(0) != rows || qi->size(1) > 64 || qi->size(2) != 64) return declined();
    }
    const at::Tensor* reserved = nullptr;
    if (a[11] != Py_None) {
      reserved = plain(a[11], at::kInt, 1, d);
      if (!reserved || reserved->size(0) != 1) return declined();
    }
    const int32_t* word = reserved ? static_cast<const int32_t*>(reserved->const_data_ptr()) : nullptr;
    dsa_rope_queries_t x = {};
    at::Tensor q_out, qi_out;
    if (q) {
      q_out = fresh({rows, q->size(1), 128}, at::kBFloat16, d);
      x.q = q->const_data_ptr();
      x.q_out = q_out.mutable_data_ptr();
      x.q_stride = qs;
      x.q_out_stride = q->size(1) * 128;
      x.Hq = static_cast<int>(q->size(1));
    }
    if (qi) {
      qi_out = fresh({rows, qi->size(1), 64}, at::kBFloat16, d);
      x.q_idx = qi->const_data_ptr();
      x.q_idx_out = qi_out.mutable_data_ptr();
      x.q_idx_stride = qis;
      x.q_idx_out_stride = qi->size(1) * 64;
      x.Hi = static_cast<int>(qi->size(1));
    }
    dsa_paged_batch_t b = *address<dsa_paged_batch_t>(a[2]);
    b.rows = rows;
    const void* cache = PyLong_AsVoidPtr(a[1]);
    const dsa_rope_t *r = address<dsa_rope_t>(a[7]), *ri = address<dsa_rope_t>(a[8]);
    const bool four = a[0] == Py_True;
    void* stream = stream_of(d);
    dsa_status_t st;
    Py_BEGIN_ALLOW_THREADS;
    st = four ? g_lib.append4(static_cast<const dsa_paged_cache4_t*>(cache), &b, k->const_data_ptr(), ks,
                              v->const_data_ptr(), vs, ki->const_data_ptr(), is, r, ri, &x, word, stream)
              : g_lib.append(static_cast<const dsa_paged_cache_t*>(cache), &b, k->const_data_ptr(), ks,
                             v->const_data_ptr(), vs, ki->const_data_ptr(), is, r, ri, &x, word, stream);
    Py_END_ALLOW_THREADS;
    if (st != DSA_OK) return PyLong_FromLong(st);
    PyObject* o1 = q ? THPVariable_Wrap(std::move(q_out)) : Py_NewRef(Py_None);
    PyObject* o2 = o1 ? (qi ? THPVariable_Wrap(std::move(qi_out)) : Py_NewRef(Py_None)) : nullptr;
    PyObject* both = o2 ? PyTuple_Pack(2, o1, o2) : nullptr;
    Py_XDECREF(o1);
    Py_XDECREF(o2);
    return both;
  });
}

// read(cache, batch, device, rows): (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const long device = n == 4 ? PyLong_AsLong(a[2]) : -1;
    const long long rows = n == 4 ? PyLong_AsLongLong(a[3]) : 0;
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return declined();
    }
    if (!takes(device) || rows < 1 || rows > (1LL << 27)) return declined();
    const int d = static_cast<int>(device);
    at::Tensor k = fresh({rows, 128}, at::kBFloat16, d), v = fresh({rows, 128}, at::kBFloat16, d);
    dsa_paged_batch_t b = *address<dsa_paged_batch_t>(a[1]);
    b.rows = rows;
    const dsa_paged_cache4_t* cache = address<dsa_paged_cache4_t>(a[0]);
    void* stream = stream_of(d);
    dsa_status_t st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_lib.read(cache, &b, k.mutable_data_ptr(), 128, v.mutable_data_ptr(), 128, stream);
    Py_END_ALLOW_THREADS;
    if (st != DSA_OK) return PyLong_FromLong(st);
    PyObject* o1 = THPVariable_Wrap(std::move(k));
    PyObject* o2 = o1 ? THPVariable_Wrap(std::move(v)) : nullptr;
    PyObject* both = o2 ? PyTuple_Pack(2, o1, o2) : nullptr;
    Py_XDECREF(o1);
    Py_XDECREF(o2);
    return both;
  });
}

// attention4(cache, batch, device, q, pool_idx, scale): (o, lse)
PyObject* attention4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6 || !(PyFloat_Check(a[5]) || PyLong_Check(a[5]))) return declined();
    const long device = PyLong_AsLong(a[2]);
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return declined();
    }
    if (!takes(device)) return declined();
    const int d = static_cast<int>(device);
    const at::Tensor *q = plain(a[3], at::kBFloat16, 3, d), *sel = plain(a[4], at::kInt, 2, d);
    if (!q || !sel || !q->is_contiguous() || !sel->is_contiguous()) return declined();
    const int64_t rows = q->size(0), hq = q->size(1), dim = q->size(2), topk = sel->size(1);
    if (rows < 1 || sel->size(0) != rows || hq > 128 || dim > 256 || topk > (1 << 20)) return declined();
    at::Tensor o = fresh({rows, hq, dim}, at::kBFloat16, d), lse = fresh({rows, hq}, at::kFloat, d);
    dsa_paged_batch_t b = *address<dsa_paged_batch_t>(a[1]);
    b.rows = rows;
    const dsa_paged_cache4_t* cache = address<dsa_paged_cache4_t>(a[0]);
    void* stream = stream_of(d);
    dsa_status_t st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_lib.attn(cache, &b, q->const_data_ptr(), static_cast<const int32_t*>(sel->const_data_ptr()),
                    static_cast<int>(hq), static_cast<int>(dim), static_cast<int>(topk), static_cast<float>(scale),
                    o.mutable_data_ptr(), static_cast<float*>(lse.mutable_data_ptr()), stream);
    Py_END_ALLOW_THREADS;
    if (st != DSA_OK) return PyLong_FromLong(st);
    PyObject* o1 = THPVariable_Wrap(std::move(o));
    PyObject* o2 = o1 ? THPVariable_Wrap(std::move(lse)) : nullptr;
    PyObject* both = o2 ? PyTuple_Pack(2, o1, o2) : nullptr;
    Py_XDECREF(o1);
    Py_XDECREF(o2);
    return both;
  });
}

// bind(rope, append, append4, read, attention4): the library's functions, as addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g_lib.rope = reinterpret_cast<RopeFn>(p[0]);
  g_lib.append = reinterpret_cast<AppendFn>(p[1]);
  g_lib.append4 = reinterpret_cast<Append4Fn>(p[2]);
  g_lib.read = reinterpret_cast<ReadFn>(p[3]);
  g_lib.attn = reinterpret_cast<AttnFn>(p[4]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attention4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", DSA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
