// binding.cpp -- the Python calls that a serving step makes, as a CPython module over the C ABI
// (include/paged_attn.h): decode, prefill, the block-scaled append and the table calls.
//
// It only turns tensors into pointers and sizes, allocates outputs that the caller did not
// give, and returns the library's status; the package's Python functions hold signatures,
// defaults and errors.  Through ctypes the same marshalling took two to three times as long
// as the call it led to (a tiny decode 20 us a call, of which the library takes 4).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <exception>

#include "paged_attn.h"

namespace {

// An argument that is not what the call takes: the Python error is set.
struct BadArgument {};

[[noreturn]] void bad(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw BadArgument();
}

const at::Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(PyExc_TypeError, "expected a tensor or None");
  return &THPVariable_Unpack(o);
}

thread_local int g_device = -1;  // the current device as this call has seen it, -1: not asked yet

void check_device(const at::Tensor& t) {
  if (!t.is_cuda()) bad(PyExc_ValueError, "tensor arguments must be CUDA tensors");
  // the library launches on the current device, whose kernels may not reach another's memory
  if (g_device < 0) g_device = c10::cuda::current_device();
  if (t.get_device() != g_device)
    bad(PyExc_ValueError, "tensor arguments must live on the current CUDA device");
}

// The device address of a contiguous CUDA tensor, null for None.
void* pointer(const at::Tensor* t) {
  if (!t) return nullptr;
  check_device(*t);
  if (!t->is_contiguous()) bad(PyExc_ValueError, "tensor arguments must be contiguous");
  return t->data_ptr();
}

void* pointer(PyObject* o) { return pointer(tensor(o)); }

const at::Tensor& required(PyObject* o, const char* what, int64_t dims) {
  const at::Tensor* t = tensor(o);
  if (!t || t->dim() != dims) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor of %lld dimensions", what, (long long)dims);
    throw BadArgument();
  }
  return *t;
}

// The address of a tensor that must have this type and at least n elements.
void* typed(const at::Tensor* t, at::ScalarType type, int64_t n, const char* what) {
  if (t && (t->scalar_type() != type || t->numel() < n)) {
    PyErr_Format(PyExc_ValueError, "%s: expected at least %lld elements of %s, got %lld of %s", what, (long long)n,
                 c10::toString(type), (long long)t->numel(), c10::toString(t->scalar_type()));
    throw BadArgument();
  }
  return pointer(t);
}

int32_t* ints(PyObject* o, int64_t n, const char* what) {
  const at::Tensor* t = tensor(o);
  if (!t) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor", what);
    throw BadArgument();
  }
  return static_cast<int32_t*>(typed(t, at::kInt, n, what));
}

int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw BadArgument();
  if (v != (int)v) bad(PyExc_OverflowError, "an integer argument does not fit 32 bits");
  return (int)v;
}

int int_of(int64_t v) {
  if (v != (int)v) bad(PyExc_OverflowError, "a tensor has more rows or elements than 32 bits count");
  return (int)v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw BadArgument();
  return v;
}

// The stream argument, None: the current stream.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw BadArgument();
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!s && PyErr_Occurred()) throw BadArgument();
  return s;
}

bool block_dtype(int kv_dtype) { return kv_dtype == PA_KV_INT8_BLOCK || kv_dtype == PA_KV_FP8_BLOCK; }

// num_pages, None: as many as the cache holds (and, for the block dtypes, at most that).
int pages_of(PyObject* num_pages, PyObject* cache, int hkv, int dqk, int dvo, int ps, int kv_dtype) {
  if (num_pages != Py_None && !block_dtype(kv_dtype)) return integer(num_pages);
  static const int x2[5] = {4, 2, 1, 2, 2};
  if (kv_dtype < 0 || kv_dtype > 4) bad(PyExc_KeyError, "unknown kv_dtype");
  const int64_t page = (int64_t)hkv * ps * (dqk + dvo) * x2[kv_dtype] / 2;
  if (page <= 0) bad(PyExc_ZeroDivisionError, "a page without bytes");
  const at::Tensor* t = tensor(cache);
  if (!t) bad(PyExc_ValueError, "kv_cache must be a tensor");
  const int64_t held = (int64_t)t->nbytes() / page;
  if (num_pages == Py_None) return int_of(held);
  const int given = integer(num_pages);
  if (given > held) bad(PyExc_ValueError, "num_pages is more than kv_cache holds");
  return given;
}

// The pointer of a block_scales pool, after checking that it covers the pages.
float* block_scales(PyObject* o, int block_tokens, int num_pages, int hkv, int ps) {
  const at::Tensor* t = tensor(o);
  if (!t || block_tokens < 1 || block_tokens > ps)
    bad(PyExc_ValueError, "the block dtypes need block_scales and 1 <= block_tokens <= page_size");
  return static_cast<float*>(typed(t, at::kFloat, (int64_t)num_pages * 2 * hkv * (ps / block_tokens), "block_scales"));
}

// The KV arguments of decode and prefill, in the order the Python functions pass them.
struct Kv {
  int hkv, dvo, ps, window, dtype, num_pages;
  float sm_scale;
  pa_kv_scales sc;
};

// a: num_kv_heads, head_dim_vo, page_size, sm_scale, window_left, kv_dtype, k_scale, v_scale,
// sf, block_scales, block_tokens, num_pages
Kv kv_of(PyObject* const* a, PyObject* cache, int dqk) {
  Kv k;
  k.hkv = integer(a[0]);
  k.dvo = integer(a[1]);
  k.ps = integer(a[2]);
  k.sm_scale = (float)real(a[3]);
  k.window = integer(a[4]);
  k.dtype = integer(a[5]);
  k.num_pages = pages_of(a[11], cache, k.hkv, dqk, k.dvo, k.ps, k.dtype);
  std::memset(&k.sc, 0, sizeof k.sc);
  if (block_dtype(k.dtype)) {
    k.sc.block_tokens = integer(a[10]);
    k.sc.block_scales = block_scales(a[9], k.sc.block_tokens, k.num_pages, k.hkv, k.ps);
  } else if (k.dtype != PA_KV_BF16) {
    k.sc.k_scale = static_cast<const float*>(pointer(a[6]));
    k.sc.v_scale = static_cast<const float*>(pointer(a[7]));
    k.sc.sf = static_cast<const uint8_t*>(pointer(a[8]));
  }
  return k;
}

struct Outputs {
  at::Tensor out, lse;
  bool has_lse;
};

// out [rows, hq, dvo] bf16 and lse [rows, hq] fp32: given, or allocated (lse if wanted)
Outputs outputs_of(PyObject* out, PyObject* lse, PyObject* return_lse, int64_t rows, int64_t hq, int64_t dvo,
                   const at::Tensor& q) {
  Outputs o;
  const at::Tensor* t = tensor(out);
  o.out = t ? *t : at::empty({rows, hq, dvo}, q.options().dtype(at::kBFloat16));
  t = tensor(lse);
  const int wanted = PyObject_IsTrue(return_lse);
  if (wanted < 0) throw BadArgument();
  o.has_lse = t || wanted;
  if (o.has_lse) o.lse = t ? *t : at::empty({rows, hq}, q.options().dtype(at::kFloat));
  return o;
}

// (status, out, lse)
PyObject* result(int status, const Outputs& o) {
  PyObject* t = PyTuple_New(3);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, PyLong_FromLong(status));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(o.out));
  PyTuple_SET_ITEM(t, 2, o.has_lse ? THPVariable_Wrap(o.lse) : Py_NewRef(Py_None));
  return t;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  g_device = -1;
  try {
    return f();
  } catch (const BadArgument&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// A library call without the interpreter lock.
template <typename F>
int call(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// decode(q, kv_cache, kv_indptr, kv_indices, kv_last_page_len, out, lse, return_lse, stream, *kv)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 21, [&]() -> PyObject* {
    const at::Tensor& q = required(a[0], "q", 3);
    const int batch = int_of(q.size(0)), hq = int_of(q.size(1)), dqk = int_of(q.size(2));
    const Kv k = kv_of(a + 9, a[1], dqk);
    void* qp = pointer(&q);
    void *cache = pointer(a[1]), *ip = pointer(a[2]), *ix = pointer(a[3]), *last = pointer(a[4]);
    const Outputs o = outputs_of(a[5], a[6], a[7], batch, hq, k.dvo, q);
    void *out = pointer(&o.out), *lse = o.has_lse ? pointer(&o.lse) : nullptr, *stream = stream_of(a[8]);
    const int st = call([&] {
      return paged_attn_decode(qp, cache, static_cast<int32_t*>(ip), static_cast<int32_t*>(ix),
                               static_cast<int32_t*>(last), batch, k.num_pages, hq, k.hkv, dqk, k.dvo, k.ps,
                               k.sm_scale, k.window, k.dtype, &k.sc, out, static_cast<float*>(lse), stream);
    });
    return result(st, o);
  });
}

// prefill(q, qo_indptr, kv_cache, kv_indptr, kv_indices, kv_last_page_len, causal, custom_mask,
//         mask_indptr, out, lse, return_lse, stream, *kv)
PyObject* py_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 25, [&]() -> PyObject* {
    const at::Tensor& q = required(a[0], "q", 3);
    const int rows = int_of(q.size(0)), hq = int_of(q.size(1)), dqk = int_of(q.size(2));
    const at::Tensor* qo = tensor(a[1]);
    if (!qo) bad(PyExc_ValueError, "qo_indptr must be a tensor");
    const int batch = int_of(qo->numel() - 1);
    const Kv k = kv_of(a + 13, a[2], dqk);
    void* qp = pointer(&q);
    void *qi = pointer(qo), *cache = pointer(a[2]), *ip = pointer(a[3]), *ix = pointer(a[4]), *last = pointer(a[5]);
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) throw BadArgument();
    const bool masked = a[7] != Py_None;
    void *mask = pointer(a[7]), *mi = pointer(a[8]);
    const Outputs o = outputs_of(a[9], a[10], a[11], rows, hq, k.dvo, q);
    void *out = pointer(&o.out), *lse = o.has_lse ? pointer(&o.lse) : nullptr, *stream = stream_of(a[12]);
    const int st = call([&] {
      if (masked)
        return paged_attn_prefill_custom_mask(
            qp, static_cast<int32_t*>(qi), rows, cache, static_cast<int32_t*>(ip), static_cast<int32_t*>(ix),
            static_cast<int32_t*>(last), batch, k.num_pages, hq, k.hkv, dqk, k.dvo, k.ps, k.sm_scale, k.window, causal,
            k.dtype, &k.sc, out, static_cast<float*>(lse), static_cast<uint8_t*>(mask), static_cast<int64_t*>(mi),
            stream);
      return paged_attn_prefill(qp, static_cast<int32_t*>(qi), rows, cache, static_cast<int32_t*>(ip),
                                static_cast<int32_t*>(ix), static_cast<int32_t*>(last), batch, k.num_pages, hq, k.hkv,
                                dqk, k.dvo, k.ps, k.sm_scale, k.window, causal, k.dtype, &k.sc, out,
                                static_cast<float*>(lse), stream);
    });
    return result(st, o);
  });
}

// append_kv_block(k_new, v_new, append_indptr, kv_cache, kv_indptr, kv_indices,
//                 kv_last_page_len, block_scales, page_size, block_tokens, kv_dtype, num_pages, stream)
PyObject* py_append_kv_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor &k = required(a[0], "k_new", 3), &v = required(a[1], "v_new", 3);
    const int total = int_of(k.size(0)), hkv = int_of(k.size(1)), dqk = int_of(k.size(2)), dvo = int_of(v.size(2));
    if (v.size(0) != total || v.size(1) != hkv || k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16)
      bad(PyExc_ValueError, "k_new and v_new must be bf16 with the same rows and kv heads");
    const at::Tensor* ai = tensor(a[2]);
    if (!ai || ai->numel() < 1) bad(PyExc_ValueError, "append_indptr must be a tensor of batch + 1 elements");
    const int batch = int_of(ai->numel() - 1);
    const int ps = integer(a[8]), bt = integer(a[9]), dtype = integer(a[10]);
    const int pages = pages_of(a[11], a[3], hkv, dqk, dvo, ps, dtype);
    void *kp = pointer(&k), *vp = pointer(&v), *cache = pointer(a[3]);
    int32_t *ap = static_cast<int32_t*>(typed(ai, at::kInt, 1, "append_indptr")),
            *ip = ints(a[4], (int64_t)batch + 1, "kv_indptr"), *ix = ints(a[5], 0, "kv_indices"),
            *last = ints(a[6], batch, "kv_last_page_len");
    float* scales = block_scales(a[7], bt, pages, hkv, ps);
    void* stream = stream_of(a[12]);
    return PyLong_FromLong(call([&] {
      return paged_attn_append_kv_block(kp, vp, ap, total, cache, ip, ix, last, batch, pages, hkv, dqk, dvo, ps, dtype,
                                        scales, bt, stream);
    }));
  });
}

struct Table {
  int32_t* p;
  int rows, width, stride;
};

// An int32 block table whose rows are contiguous.
Table table_of(PyObject* o) {
  const at::Tensor* t = tensor(o);
  if (t) check_device(*t);
  if (!t || t->scalar_type() != at::kInt || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1))
    bad(PyExc_ValueError, "block_table must be int32 [rows, max_pages] with contiguous rows");
  return {static_cast<int32_t*>(t->data_ptr()), int_of(t->size(0)), int_of(t->size(1)),
          int_of(std::max(t->stride(0), t->size(1)))};
}

int32_t* row_ids_of(PyObject* o, int batch) { return o == Py_None ? nullptr : ints(o, batch, "row_ids"); }

// resize_tables(block_table, row_ids, kv_lens, deltas, free_pages, free_count, page_size, stream)
PyObject* py_resize_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Table t = table_of(a[0]);
    int32_t* deltas = ints(a[3], 0, "deltas");
    const int batch = int_of(tensor(a[3])->numel());
    int32_t *ids = row_ids_of(a[1], batch), *lens = ints(a[2], t.rows, "kv_lens"), *free = ints(a[4], 0, "free_pages"),
            *count = ints(a[5], 1, "free_count");
    const int size = int_of(tensor(a[4])->numel()), ps = integer(a[6]);
    void* stream = stream_of(a[7]);
    return PyLong_FromLong(call([&] {
      return paged_attn_resize_tables(t.p, t.rows, t.width, t.stride, ids, lens, deltas, batch, ps, free, size, count,
                                      stream);
    }));
  });
}

// build_tables(block_table, row_ids, kv_lens, new_counts, page_size, num_pages, max_indices,
//              num_tokens, out, stream) -> (status, out); out None: allocated
PyObject* py_build_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Table t = table_of(a[0]);
    int32_t* counts = ints(a[3], 0, "new_counts");
    const int batch = int_of(tensor(a[3])->numel());
    int32_t *ids = row_ids_of(a[1], batch), *lens = ints(a[2], t.rows, "kv_lens");
    const int ps = integer(a[4]), pages = integer(a[5]), most = integer(a[6]), tokens = integer(a[7]);
    if (most < 0 || tokens < 0) bad(PyExc_ValueError, "max_indices and num_tokens must not be negative");
    at::Tensor o[6];
    const int64_t sizes[6] = {(int64_t)batch + 1, most, batch, (int64_t)batch + 1, tokens, tokens};
    static const char* const names[6] = {"kv_indptr", "kv_indices", "kv_last_page_len", "new_indptr", "slot_map",
                                         "positions"};
    void* ptr[6];
    if (a[8] != Py_None && (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 6))
      bad(PyExc_ValueError, "out must be a tuple of six tensors");
    for (int i = 0; i < 6; ++i) {
      const at::ScalarType type = i == 4 ? at::kLong : at::kInt;
      if (a[8] == Py_None) {
        o[i] = at::empty({sizes[i]}, tensor(a[0])->options().dtype(type));
      } else {
        const at::Tensor* given = tensor(PyTuple_GET_ITEM(a[8], i));
        if (!given) bad(PyExc_ValueError, "out must be a tuple of six tensors");
        o[i] = *given;
      }
      ptr[i] = typed(&o[i], type, sizes[i], names[i]);
    }
    void* stream = stream_of(a[9]);
    const int st = call([&] {
      auto i32 = [&](int i) { return static_cast<int32_t*>(ptr[i]); };
      return paged_attn_build_tables(t.p, t.rows, t.width, t.stride, ids, lens, counts, batch, ps, pages, i32(0),
                                     i32(1), most, i32(2), i32(3), static_cast<int64_t*>(ptr[4]), i32(5), tokens,
                                     stream);
    });
    PyObject* r = PyTuple_New(6);
    if (!r) return nullptr;
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(o[i]));
    return Py_BuildValue("(iN)", st, r);
  });
}

PyMethodDef methods[] = {{"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, nullptr},
                         {"prefill", (PyCFunction)(void (*)(void))py_prefill, METH_FASTCALL, nullptr},
                         {"append_kv_block", (PyCFunction)(void (*)(void))py_append_kv_block, METH_FASTCALL, nullptr},
                         {"resize_tables", (PyCFunction)(void (*)(void))py_resize_tables, METH_FASTCALL, nullptr},
                         {"build_tables", (PyCFunction)(void (*)(void))py_build_tables, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
