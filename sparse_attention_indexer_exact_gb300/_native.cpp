// _native.cpp -- the short way from torch tensors to the C ABI of include/gvr_cache.h.
//
// A call of cache.py costs the host more than the GPU needs for the smallest ones, nearly all of it in
// reading tensor properties from Python.  The functions here read them directly, make the call and
// return its results, or return None where anything is out of the ordinary: a wrong type or shape,
// another device than the current one, a refusal by the library.  cache.py then takes its own way,
// which does the same step by step and raises the error that names what is wrong.  Measured on a
// GB300's host: 20 us a call of attend_decode through Python and ctypes, 3.9 this way (1.9 without outputs to
// allocate).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "gvr_cache.h"

namespace {

using at::Tensor;

// Thrown where the Python way has to be taken; it never leaves this file.
struct Otherwise {};

inline void need(bool ok) {
  if (!ok) throw Otherwise{};
}

const Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  need(PyLong_CheckExact(o));
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  need(!overflow);
  return v;
}

int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  need(v >= INT32_MIN && v <= INT32_MAX);
  return int32_t(v);
}

float number(PyObject* o) {
  need(PyFloat_CheckExact(o));
  return float(PyFloat_AS_DOUBLE(o));
}

// The current device and its stream; every tensor of a call has to be on it.
struct Where {
  c10::DeviceIndex device = c10::cuda::current_device();
  void* stream = c10::cuda::getCurrentCUDAStream(device).stream();

  const Tensor& on(const Tensor& t, at::ScalarType type) const {
    need(t.is_cuda() && t.device().index() == device && t.scalar_type() == type && t.layout() == at::kStrided);
    return t;
  }
  // From torch's allocator on the current stream, without the dispatcher (1.1 -> 0.6 us each).
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_generic(size, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                     std::nullopt);
  }
};

// A contiguous 1-D int32 tensor of at least `least` entries.
const int32_t* int32s(const Where& w, const Tensor& t, int64_t least) {
  w.on(t, at::kInt);
  need(t.dim() == 1 && t.size(0) >= least && (t.size(0) <= 1 || t.stride(0) == 1));
  return static_cast<const int32_t*>(t.data_ptr());
}

int32_t dtype_of(const Tensor& t) {
  need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf);
  return t.scalar_type() == at::kBFloat16 ? GVR_BF16 : GVR_F16;
}

struct Heads {
  const void* data;
  int64_t row, head;
};

Heads heads_of(const Where& w, const Tensor& t, int64_t dim) {
  w.on(t, t.scalar_type());
  need(t.dim() == 3 && t.size(2) == dim);
  if (t.numel() == 0) return {t.data_ptr(), 0, 0};
  need(t.stride(2) == 1);
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

struct Table {
  int32_t* data;
  int64_t stride, width, rows;
};

Table table_of(const Where& w, const Tensor& t, int64_t requests) {
  w.on(t, at::kInt);
  need(t.dim() == 2 && t.size(0) >= requests && (t.size(0) == 0 || t.size(1) <= 1 || t.stride(1) == 1));
  return {static_cast<int32_t*>(t.data_ptr()), t.size(0) > 1 ? t.stride(0) : t.size(1), t.size(1), t.size(0)};
}

gvr_cache cache_of(const Where& w, const Tensor& t, float k_scale, float v_scale) {
  w.on(t, at::kByte);
  need(t.dim() == 4);
  const int64_t pages = t.size(0), size = t.size(1), heads = t.size(2), row = t.size(3);
  const int32_t dim = row == 80 ? 64 : row == 144 ? 128 : row == 288 ? 256 : 0;
  need(dim != 0 && size <= INT32_MAX && heads <= INT32_MAX);
  need(pages == 0 || (t.stride(3) == 1 && (heads <= 1 || t.stride(2) == row) && (size <= 1 || t.stride(1) == heads * row)));
  return {t.data_ptr(), pages, pages > 1 ? t.stride(0) : size * heads * row, int32_t(size), int32_t(heads), dim, 0, k_scale, v_scale};
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// (cached_lens, kv_lens, free_pages, block_table, max_new, page_size, compress_ratio, slots, counts)
PyObject* tables(PyObject* const* a) {
  const Where w;
  const Tensor &cached = tensor(a[0]), &lens = tensor(a[1]), &free_pages = tensor(a[2]);
  need(lens.dim() == 1);
  const int64_t requests = lens.size(0), max_new = integer(a[4]);
  const int32_t *lens_at = int32s(w, lens, 0), *cached_at = int32s(w, cached, requests), *free_at = int32s(w, free_pages, 0);
  const Table table = table_of(w, tensor(a[3]), requests);
  const int32_t page_size = integer32(a[5]), ratio = integer32(a[6]);
  need(max_new >= 0);
  const Tensor slots = a[7] == Py_None ? w.empty({max_new}, at::kInt) : tensor(a[7]);
  const Tensor counts = a[8] == Py_None ? w.empty({3}, at::kInt) : tensor(a[8]);
  int32_t *slots_at = const_cast<int32_t*>(int32s(w, slots, max_new)), *counts_at = const_cast<int32_t*>(int32s(w, counts, 3));
  need(cache_tables(cached_at, lens_at, requests, ratio, page_size, free_at, free_pages.size(0), table.data, table.stride,
                    table.width, slots_at, max_new, counts_at, w.stream) == GVR_OK);
  return pair(slots, counts);
}

// (k, v, cache, slots, k_scale, v_scale)
PyObject* append(PyObject* const* a) {
  const Where w;
  const Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  const gvr_cache c = cache_of(w, tensor(a[2]), number(a[4]), number(a[5]));
  const int32_t kind = dtype_of(k);
  need(v.scalar_type() == k.scalar_type() && v.sizes() == k.sizes());
  const Heads kh = heads_of(w, k, c.head_dim), vh = heads_of(w, v, c.head_dim);
  need(k.size(1) == c.num_kv_heads);
  const int32_t* slots = int32s(w, tensor(a[3]), k.size(0));
  need(cache_append(&c, kh.data, kh.row, kh.head, vh.data, vh.row, vh.head, kind, slots, k.size(0), w.stream) == GVR_OK);
  Py_RETURN_TRUE;
}

// (cache, slots, head_dim, kind, k_scale, v_scale): kind is the wanted type, as in gvr_cache.h
PyObject* read(PyObject* const* a) {
  const Where w;
  const gvr_cache c = cache_of(w, tensor(a[0]), number(a[4]), number(a[5]));
  const Tensor& slots = tensor(a[1]);
  need(c.head_dim == integer(a[2]));
  const int32_t kind = integer32(a[3]);
  need(kind == GVR_BF16 || kind == GVR_F16);
  const int32_t* at = int32s(w, slots, 0);
  const int64_t n = slots.size(0);
  const at::ScalarType type = kind == GVR_BF16 ? at::kBFloat16 : at::kHalf;
  const Tensor k = w.empty({n, c.num_kv_heads, c.head_dim}, type), v = w.empty({n, c.num_kv_heads, c.head_dim}, type);
  need(cache_read(&c, at, n, kind, k.data_ptr(), v.data_ptr(), w.stream) == GVR_OK);
  return pair(k, v);
}

struct Attend {
  gvr_cache c;
  Heads q;
  int32_t kind;
  int64_t rows, heads;
  float scale;
  Tensor out, lse;
  void* lse_at;

  // q, cache, k_scale, v_scale, scale, out, lse, want_lse
  Attend(const Where& w, PyObject* const* a) {
    const Tensor& t = tensor(a[0]);
    c = cache_of(w, tensor(a[1]), number(a[2]), number(a[3]));
    kind = dtype_of(t);
    q = heads_of(w, t, c.head_dim);
    rows = t.size(0), heads = t.size(1);
    need(heads > 0 && heads <= INT32_MAX && c.num_kv_heads > 0 && heads % c.num_kv_heads == 0);
    scale = a[4] == Py_None ? float(1.0 / std::sqrt(double(c.head_dim))) : number(a[4]);
    if (a[5] == Py_None) {
      out = w.empty({rows, heads, c.head_dim}, t.scalar_type());
    } else {
      out = w.on(tensor(a[5]), t.scalar_type());
      need(out.sizes() == t.sizes() && out.is_contiguous());
    }
    if (a[6] != Py_None) {
      lse = w.on(tensor(a[6]), at::kFloat);
      need(lse.dim() == 2 && lse.size(0) == rows && lse.size(1) == heads && lse.is_contiguous());
    } else {
      need(a[7] == Py_True || a[7] == Py_False);
      if (a[7] == Py_True) lse = w.empty({rows, heads}, at::kFloat);
    }
    lse_at = lse.defined() ? lse.data_ptr() : nullptr;
  }
};

struct Listed {
  const int32_t* data = nullptr;
  int64_t k = 0;
  Tensor workspace;

  Listed(const Where& w, PyObject* indices, int64_t rows) {
    if (indices != Py_None) {
      const Tensor& t = w.on(tensor(indices), at::kInt);
      need(t.dim() == 2 && t.size(0) == rows && t.size(1) >= 1 && t.is_contiguous());
      data = static_cast<const int32_t*>(t.data_ptr()), k = t.size(1);
    }
    if (k == 0 || k > LONG) workspace = w.empty({GVR_ATTEND_WORKSPACE}, at::kByte);
  }
  void* at() const { return workspace.defined() ? workspace.data_ptr() : nullptr; }

  static constexpr int64_t LONG = 2048;  // as in cache.py
};

// (q, cache, k_scale, v_scale, scale, out, lse, want_lse, block_table, kv_lens, next_n, compress_ratio, indices)
PyObject* decode(PyObject* const* a) {
  const Where w;
  const Attend x(w, a);
  const int32_t next_n = integer32(a[10]), ratio = integer32(a[11]);
  need(next_n >= 1);
  const int64_t requests = (x.rows + next_n - 1) / next_n;
  const Table t = table_of(w, tensor(a[8]), requests);
  const int32_t* lens = int32s(w, tensor(a[9]), requests);
  const Listed l(w, a[12], x.rows);
  need(attend_decode(&x.c, x.q.data, x.q.row, x.q.head, x.kind, x.rows, int32_t(x.heads), t.data, t.stride, t.width, lens, next_n,
                     ratio, l.data, l.k, x.scale, x.out.data_ptr(), static_cast<float*>(x.lse_at), l.at(),
                     GVR_ATTEND_WORKSPACE, w.stream) == GVR_OK);
  return pair(x.out, x.lse);
}

// (q, cache, k_scale, v_scale, scale, out, lse, want_lse, block_table, row_requests, row_starts, row_ends, indices)
PyObject* prefill(PyObject* const* a) {
  const Where w;
  const Attend x(w, a);
  const Table t = table_of(w, tensor(a[8]), 0);
  const int32_t *requests = int32s(w, tensor(a[9]), x.rows), *starts = int32s(w, tensor(a[10]), x.rows), *ends = int32s(w, tensor(a[11]), x.rows);
  const Listed l(w, a[12], x.rows);
  need(l.data != nullptr);
  need(attend_prefill(&x.c, x.q.data, x.q.row, x.q.head, x.kind, x.rows, int32_t(x.heads), t.data, t.stride, t.width, t.rows,
                      requests, starts, ends, l.data, l.k, x.scale, x.out.data_ptr(), static_cast<float*>(x.lse_at), l.at(),
                      GVR_ATTEND_WORKSPACE, w.stream) == GVR_OK);
  return pair(x.out, x.lse);
}

template <PyObject* (*call)(PyObject* const*), int arguments>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n == arguments) {
    try {
      at::AutoDispatchBelowADInplaceOrView guard;
      if (PyObject* r = call(args)) return r;
    } catch (...) {  // Otherwise, or an error of torch's that the Python way meets again
    }
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <PyObject* (*call)(PyObject* const*), int arguments>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<call, arguments>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<tables, 9>("cache_tables"), method<append, 6>("cache_append"), method<read, 6>("cache_read"),
                         method<decode, 13>("attend_decode"), method<prefill, 13>("attend_prefill"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "The short way from tensors to the cache kernels.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// BUILT_FOR is compared before the first call: under another torch nothing here may be used.
PyMODINIT_FUNC PyInit__native() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", GVR_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
