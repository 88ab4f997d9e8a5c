// The short way into the decoding calls (rotary positions and the 4-bit
// cache): a CPython module that checks the tensors of one call, allocates its
// outputs and calls the C ABI, in about 2 us plus the launch.  A decoding step
// makes these calls once per layer and their kernels run for 4 to 20 us, which
// the same work in Python (6 to 14 us a call) would not keep up with.
//
// Every function answers None for whatever is not plainly right: another type,
// shape or layout than the usual ones, a tensor on another device than the
// current one, an argument it does not know.  The caller then takes the long
// way, whose checks say what is wrong, or serve the rarer forms.  Nothing is
// launched before all checks have passed.  A call that the C ABI refuses gives
// its status code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>

#include "kvz.h"

namespace {

struct Calls {
  decltype(&kvz_rotary) rotary = nullptr;
  decltype(&kvz_compact_int4) compact = nullptr;
  decltype(&kvz_append_int4) append = nullptr;
  decltype(&kvz_expand_int4) expand = nullptr;
  decltype(&kvz_decode_int4) decode = nullptr;
  decltype(&kvz_decode_int4_workspace_size) decode_size = nullptr;
} g;

// One call's arguments: any failed check clears `ok`.
struct Args {
  bool ok = true;
  int dev = -1;

  // A CUDA tensor of the type on the call's device; null for None (if it may be) or a failure.
  const at::Tensor* tensor(PyObject* o, at::ScalarType type, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!ok || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.layout() != at::kStrided) return fail();
    const int d = t.get_device();
    if (dev < 0) dev = d;
    if (d != dev) return fail();
    return &t;
  }
  const at::Tensor* dense(PyObject* o, at::ScalarType type, int64_t numel, bool optional = false) {
    const at::Tensor* t = tensor(o, type, optional);
    if (t != nullptr && (t->numel() < numel || !t->is_contiguous())) return fail();
    return t;
  }
  const at::Tensor* dense_as(PyObject* o, at::ScalarType type, at::IntArrayRef shape, bool optional = false) {
    const at::Tensor* t = tensor(o, type, optional);
    if (t != nullptr && (t->sizes() != shape || !t->is_contiguous())) return fail();
    return t;
  }
  // bf16 rows: dense last dimension, other strides multiples of 8, 16-byte aligned.
  const at::Tensor* rows(PyObject* o, int64_t dims) {
    const at::Tensor* t = tensor(o, at::kBFloat16);
    if (t == nullptr) return nullptr;
    if (t->dim() != dims || t->stride(dims - 1) != 1 || (reinterpret_cast<uintptr_t>(t->const_data_ptr()) & 15) != 0)
      return fail();
    for (int64_t i = 0; i + 1 < dims; ++i)
      if (t->stride(i) % 8 != 0) return fail();
    return t;
  }
  int64_t integer(PyObject* o) {
    if (!PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred() != nullptr) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int flag(PyObject* o) {
    if (o != Py_True && o != Py_False) ok = false;
    return o == Py_True ? 1 : 0;
  }
  bool current() const { return ok && dev >= 0 && c10::cuda::current_device() == dev; }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }
  // (through the dispatcher a call with two outputs takes 0.5 us more, 5.3 against 4.8; where torch was asked to fill
  // new memory, what no call writes is filled as torch.empty does)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const at::Context& ctx = at::globalContext();
    if (ctx.deterministicAlgorithms() && ctx.deterministicFillUninitializedMemory())
      return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                             std::nullopt));
  }

 private:
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

template <class T>
T* ptr(const at::Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}

// A page pool and table: cache uint8 [n_pages, page_size * d * 9 / 8], pages int32 [B, max_pages].
struct Pages {
  const at::Tensor* cache;
  const at::Tensor* pages;
  int64_t page_size;
  bool take(Args& a, PyObject* cache_o, PyObject* pages_o, PyObject* page_size_o) {
    cache = a.dense(cache_o, at::kByte, 1);
    pages = a.dense(pages_o, at::kInt, 1);
    page_size = a.integer(page_size_o);
    return a.ok && cache->dim() == 2 && pages->dim() == 2 && page_size >= 16 && page_size <= 1024 &&
           page_size % 16 == 0;
  }
  bool fits(int64_t B, int64_t d) const {
    return (d == 64 || d == 128) && cache->size(1) * 8 == page_size * d * 9 && pages->size(0) == B;
  }
};

// Positions int32 [n] or [B, n] and table fp32 [n_pos, rot].
struct Turn {
  const at::Tensor* pos = nullptr;
  const at::Tensor* table = nullptr;
  int64_t sb = 0;
  bool take(Args& a, PyObject* pos_o, PyObject* table_o, int64_t B, int64_t n) {
    pos = a.dense(pos_o, at::kInt, 1);
    table = a.dense(table_o, at::kFloat, 1);
    if (!a.ok || table->dim() != 2) return false;
    if (pos->dim() == 1 && pos->size(0) == n) sb = 0;
    else if (pos->dim() == 2 && pos->size(0) == B && pos->size(1) == n) sb = n;
    else return false;
    return true;
  }
};

// Tensors of one allocation may overlap: the long way looks closer.
bool same_memory(const at::Tensor& x, const at::Tensor& y) {
  return x.storage().unsafeGetStorageImpl() == y.storage().unsafeGetStorageImpl();
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* done(kvz_status st, PyObject* result) {
  if (st == KVZ_OK) return result;
  Py_XDECREF(result);
  return PyLong_FromLong(st);
}
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* pair(PyObject* a, PyObject* b) {                   // takes both references
  PyObject* t = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  return t;
}

// An at:: call that throws (out of memory) becomes the Python error it stands for.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const c10::OutOfMemoryError& e) {
    // the long way raises it as torch does
    return none();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// rotary(x, positions, table, interleaved, inverse, status)
PyObject* rotary(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 6 || g.rotary == nullptr) return none();
  return guarded([&]() -> PyObject* {
    Args a;
    if (!THPVariable_Check(v[0])) return none();
    const int64_t dims = THPVariable_Unpack(v[0]).dim();
    if (dims != 3 && dims != 4) return none();
    const at::Tensor* x = a.rows(v[0], dims);
    if (!a.ok || x->numel() == 0) return none();
    const bool grouped = dims == 4;
    const int64_t B = x->size(0), G = grouped ? x->size(1) : 1, T = x->size(dims - 2), d = x->size(dims - 1);
    Turn t;
    if (!t.take(a, v[1], v[2], B, T)) return none();
    const int il = a.flag(v[3]), inv = a.flag(v[4]);
    const at::Tensor* status = a.dense(v[5], at::kInt, 1, true);
    if (!a.current() || G > 65535) return none();
    const at::Tensor y = a.empty(x->sizes(), at::kBFloat16);
    const kvz_status st = g.rotary(x->const_data_ptr(), x->stride(0), grouped ? x->stride(1) : 0, x->stride(dims - 2), B,
                                   static_cast<int>(G), T, static_cast<int>(d), ptr<int32_t>(t.pos), t.sb,
                                   ptr<float>(t.table), t.table->size(0), static_cast<int>(t.table->size(1)), il, inv,
                                   y.data_ptr(), G * T * d, T * d, d, ptr<int32_t>(status), a.stream());
    return done(st, THPVariable_Wrap(y));
  });
}

// compact(K, V, idx, counts, offsets, cache, pages, page_size, status)
PyObject* compact(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 9 || g.compact == nullptr) return none();
  return guarded([&]() -> PyObject* {
    Args a;
    const at::Tensor* K = a.dense(v[0], at::kBFloat16, 1);
    const at::Tensor* V = a.dense(v[1], at::kBFloat16, 1);
    if (!a.ok || K->dim() != 3 || V->sizes() != K->sizes()) return none();
    const int64_t B = K->size(0), d = K->size(2);
    const at::Tensor* idx = a.dense(v[2], at::kInt, 1);
    const at::Tensor* counts = a.dense(v[3], at::kInt, B);
    const at::Tensor* offsets = a.dense(v[4], at::kLong, B + 1);
    Pages pg;
    if (!pg.take(a, v[5], v[6], v[7]) || !pg.fits(B, d)) return none();
    const at::Tensor* status = a.dense(v[8], at::kInt, 1, true);
    if (!a.current()) return none();
    const kvz_status st = g.compact(K->const_data_ptr(), V->const_data_ptr(), B, K->size(1), static_cast<int>(d),
                                    ptr<int32_t>(idx), ptr<int32_t>(counts), ptr<int64_t>(offsets),
                                    pg.cache->data_ptr(), pg.cache->size(0), static_cast<int>(pg.page_size),
                                    ptr<int32_t>(pg.pages), pg.pages->size(1), ptr<int32_t>(status), a.stream());
    return done(st, given(v[5]));
  });
}

// append(k, v, cache, pages, counts, page_size, positions, table, interleaved, q, q_out, n_new, counts_out, status)
PyObject* append(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 14 || g.append == nullptr) return none();
  return guarded([&]() -> PyObject* {
    Args a;
    const at::Tensor* k = a.rows(v[0], 3);
    const at::Tensor* x = a.rows(v[1], 3);
    if (!a.ok || k->numel() == 0 || x->sizes() != k->sizes()) return none();
    const int64_t B = k->size(0), T = k->size(1), d = k->size(2);
    Pages pg;
    if (!pg.take(a, v[2], v[3], v[5]) || !pg.fits(B, d)) return none();
    const at::Tensor* counts = a.dense(v[4], at::kInt, B);
    Turn t;
    if ((v[6] != Py_None || v[7] != Py_None) && !t.take(a, v[6], v[7], B, T)) return none();
    const int il = a.flag(v[8]);
    const at::Tensor* q = nullptr;
    const at::Tensor* q_given = nullptr;
    int64_t G = 1;
    if (v[9] != Py_None) {
      q = a.rows(v[9], 4);
      if (!a.ok || q->size(0) != B || q->size(2) != T || q->size(3) != d) return none();
      G = q->size(1);
      q_given = a.dense_as(v[10], at::kBFloat16, {B, G, T, d}, true);
      if (!a.ok || G < 1 || G > 65535) return none();
      if (q_given != nullptr && same_memory(*q_given, *q)) return none();
    } else if (v[10] != Py_None) {
      return none();
    }
    const at::Tensor* n_new = a.dense(v[11], at::kInt, B, true);
    const at::Tensor* n_out = a.dense(v[12], at::kInt, B, true);
    const at::Tensor* status = a.dense(v[13], at::kInt, 1, true);
    if (!a.current()) return none();
    if (n_out != nullptr && (same_memory(*n_out, *counts) || (n_new != nullptr && same_memory(*n_out, *n_new)) ||
                             (t.pos != nullptr && same_memory(*n_out, *t.pos))))
      return none();
    if (q_given != nullptr && (same_memory(*q_given, *k) || same_memory(*q_given, *x))) return none();
    at::Tensor n_empty;
    if (n_out == nullptr) n_empty = a.empty({B}, at::kInt);
    at::Tensor q_new;
    if (q != nullptr && q_given == nullptr) q_new = a.empty({B, G, T, d}, at::kBFloat16);
    void* const qo = q == nullptr ? nullptr : (q_given != nullptr ? q_given->data_ptr() : q_new.data_ptr());
    const kvz_status st = g.append(
        k->const_data_ptr(), k->stride(0), k->stride(1), x->const_data_ptr(), x->stride(0), x->stride(1),
        q == nullptr ? nullptr : q->const_data_ptr(), q == nullptr ? 0 : q->stride(0), q == nullptr ? 0 : q->stride(1),
        q == nullptr ? 0 : q->stride(2), qo, B, static_cast<int>(G), T, static_cast<int>(d), ptr<int32_t>(t.pos), t.sb,
        ptr<float>(t.table), t.table == nullptr ? 0 : t.table->size(0),
        t.table == nullptr ? 0 : static_cast<int>(t.table->size(1)), il, pg.cache->data_ptr(), pg.cache->size(0),
        static_cast<int>(pg.page_size), ptr<int32_t>(pg.pages), pg.pages->size(1), ptr<int32_t>(counts),
        ptr<int32_t>(n_new), ptr<int32_t>(n_out != nullptr ? n_out : &n_empty), ptr<int32_t>(status), a.stream());
    PyObject* const second =
        q == nullptr ? given(Py_None) : (q_given != nullptr ? given(v[10]) : THPVariable_Wrap(q_new));
    return done(st, pair(n_out != nullptr ? given(v[12]) : THPVariable_Wrap(n_empty), second));
  });
}

// expand(cache, pages, counts, offsets, page_size, first, out_rows, status)
PyObject* expand(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 8 || g.expand == nullptr) return none();
  return guarded([&]() -> PyObject* {
    Args a;
    Pages pg;
    if (!pg.take(a, v[0], v[1], v[4])) return none();
    const int64_t B = pg.pages->size(0), d = pg.cache->size(1) == pg.page_size * 144 ? 128 : 64;
    if (!pg.fits(B, d)) return none();
    const at::Tensor* counts = a.dense(v[2], at::kInt, B);
    const at::Tensor* offsets = a.dense(v[3], at::kLong, B + 1);
    const at::Tensor* first = a.dense(v[5], at::kInt, B, true);
    const int64_t rows = a.integer(v[6]);
    const at::Tensor* status = a.dense(v[7], at::kInt, 1, true);
    if (!a.current() || rows < 1) return none();
    const at::Tensor K = a.empty({rows, d}, at::kBFloat16), V = a.empty({rows, d}, at::kBFloat16);
    const kvz_status st = g.expand(pg.cache->const_data_ptr(), pg.cache->size(0), static_cast<int>(pg.page_size),
                                   ptr<int32_t>(pg.pages), pg.pages->size(1), ptr<int32_t>(counts), ptr<int32_t>(first),
                                   ptr<int64_t>(offsets), B, static_cast<int>(d), K.data_ptr(), V.data_ptr(), rows,
                                   ptr<int32_t>(status), a.stream());
    return done(st, pair(THPVariable_Wrap(K), THPVariable_Wrap(V)));
  });
}

// decode(q, cache, pages, counts, page_size, scale, out, lse2, workspace, status)
PyObject* decode(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 10 || g.decode == nullptr) return none();
  return guarded([&]() -> PyObject* {
    Args a;
    const at::Tensor* q = a.dense(v[0], at::kBFloat16, 1);
    if (!a.ok || q->dim() != 3) return none();
    const int64_t B = q->size(0), G = q->size(1), d = q->size(2);
    Pages pg;
    if (!pg.take(a, v[1], v[2], v[4]) || !pg.fits(B, d)) return none();
    const at::Tensor* counts = a.dense(v[3], at::kInt, B);
    if ((v[5] != Py_None && !PyFloat_Check(v[5])) || G > 8) return none();
    const float scale = static_cast<float>(v[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d))
                                                           : PyFloat_AS_DOUBLE(v[5]));
    const at::Tensor* out_given = a.dense_as(v[6], at::kFloat, {B, G, d}, true);
    const at::Tensor* lse_given = a.dense_as(v[7], at::kFloat, {B, G}, true);
    const at::Tensor* ws_given = a.dense(v[8], at::kByte, 0, true);
    const at::Tensor* status = a.dense(v[9], at::kInt, 1, true);
    if (!a.current()) return none();
    at::Tensor out, lse, ws;
    if (out_given == nullptr) out = a.empty({B, G, d}, at::kFloat);
    if (lse_given == nullptr) lse = a.empty({B, G}, at::kFloat);
    void* w = ptr<void>(ws_given);
    size_t w_bytes = ws_given == nullptr ? 0 : static_cast<size_t>(ws_given->numel());
    if (ws_given == nullptr) {
      w_bytes = g.decode_size(B, static_cast<int>(G), pg.pages->size(1) * pg.page_size, static_cast<int>(d));
      if (w_bytes > 0) {
        ws = a.empty({static_cast<int64_t>(w_bytes)}, at::kByte);
        w = ws.data_ptr();
      }
    }
    const kvz_status st = g.decode(q->const_data_ptr(), pg.cache->const_data_ptr(), pg.cache->size(0),
                                   static_cast<int>(pg.page_size), ptr<int32_t>(pg.pages), pg.pages->size(1),
                                   ptr<int32_t>(counts), B, static_cast<int>(G), static_cast<int>(d), scale,
                                   out_given != nullptr ? ptr<float>(out_given) : ptr<float>(&out),
                                   lse_given != nullptr ? ptr<float>(lse_given) : ptr<float>(&lse), w, w_bytes,
                                   ptr<int32_t>(status), a.stream());
    return done(st, pair(out_given != nullptr ? given(v[6]) : THPVariable_Wrap(out),
                         lse_given != nullptr ? given(v[7]) : THPVariable_Wrap(lse)));
  });
}

// bind(address of kvz_rotary, compact, append, expand, decode, decode's workspace size)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  void* at[6];
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(v[i]);
    if (at[i] == nullptr) return PyErr_Occurred() != nullptr ? nullptr : none();
  }
  g.rotary = reinterpret_cast<decltype(g.rotary)>(at[0]);
  g.compact = reinterpret_cast<decltype(g.compact)>(at[1]);
  g.append = reinterpret_cast<decltype(g.append)>(at[2]);
  g.expand = reinterpret_cast<decltype(g.expand)>(at[3]);
  g.decode = reinterpret_cast<decltype(g.decode)>(at[4]);
  g.decode_size = reinterpret_cast<decltype(g.decode_size)>(at[5]);
  return none();
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},       {"rotary", fast(rotary), METH_FASTCALL, nullptr},
    {"compact", fast(compact), METH_FASTCALL, nullptr}, {"append", fast(append), METH_FASTCALL, nullptr},
    {"expand", fast(expand), METH_FASTCALL, nullptr},   {"decode", fast(decode), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvz_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvz_fast(void) {
  PyObject* const m = PyModule_Create(&module);
  if (m != nullptr && (PyModule_AddStringConstant(m, "torch_version", KVZ_TORCH_VERSION) != 0 ||
                       PyModule_AddStringConstant(m, "header_id", KVZ_HEADER_ID) != 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
