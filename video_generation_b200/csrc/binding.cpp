// binding.cpp -- marshalling of tensors for the attention-layer operators of
// libaf (include/af.h), as the CPython module video_generation_b200._binding.
//
// A call on one token takes 2 to 5 us on the GPU; checking six tensors and
// making the outputs in Python took 15 us (ctypes 2 of them).  Measured now: 2.3
// to 2.9 us of host time a call with the launch, 4.5 with two outputs to make.
// The functions check shapes, types, strides and devices, make outputs that
// are not given, and call the library.  They return the outputs, or the
// library's status as an int when it is not AF_OK; a tensor that cannot be
// passed on raises ValueError.  None of the calls has a gradient: a tensor that
// autograd follows is refused, and what a call writes moves its version counter.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/af.h"

namespace {

decltype(&::af_qk_norm_rope) p_qk;
decltype(&::af_cache_write) p_write;
decltype(&::af_cache_read) p_read;
decltype(&::af_cache_attention) p_attn;
decltype(&::af_cache_attention_workspace_bytes) p_ws;
decltype(&::af_cache_bytes) p_bytes;

// What ends a call as a Python ValueError.
[[noreturn]] void bad(const std::string& msg) { throw std::invalid_argument(msg); }
struct PyFailed {};   // a Python error is set already

const at::Tensor* tensor(const char* what, PyObject* o, bool optional) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(what) + ": not a tensor");
  const at::Tensor* t = &THPVariable_Unpack(o);
  if (c10::GradMode::is_enabled() && t->requires_grad())
    bad(std::string(what) + ": a tensor that requires grad, and the call has no gradient: make it under torch.no_grad(), or of detached tensors");
  return t;
}
// The caller's tensor was written behind autograd's back: a graph that saved it must not use it.
void written(const at::Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
void on_device(const char* what, const at::Tensor* t, int dev) {
  if (t && (!t->is_cuda() || t->get_device() != dev))
    bad(std::string(what) + ": a tensor on " + t->device().str() + ", the current device is cuda:" + std::to_string(dev));
}
std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

// The row stride of [..., rows, heads, dim] whose heads are consecutive slices of a row.
int64_t row_stride(const char* what, const at::Tensor& t, int64_t heads, int64_t dim, at::ScalarType type) {
  const int64_t n = t.dim();
  if (n < 3 || t.scalar_type() != type || t.size(n - 2) != heads || t.size(n - 1) != dim)
    bad(std::string(what) + ": " + c10::toString(type) + " [..., " + std::to_string(heads) + ", " + std::to_string(dim) +
        "], got " + c10::toString(t.scalar_type()) + " " + shape_of(t));
  if (t.numel() && (t.stride(n - 1) != 1 || (heads > 1 && t.stride(n - 2) != dim)))
    bad(std::string(what) + ": a row's heads must be consecutive");
  return t.size(n - 3) > 1 ? t.stride(n - 3) : heads * dim;
}
int64_t batch_stride(const at::Tensor& t, int64_t row) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * row; }

const int32_t* ints(const char* what, const at::Tensor* t, int64_t n, int64_t m = 0) {
  if (!t) return nullptr;
  const bool shape = m ? t->dim() == 2 && t->size(0) == n && t->size(1) == m : t->dim() == 1 && t->size(0) == n;
  if (t->scalar_type() != at::kInt || !shape || !t->is_contiguous())
    bad(std::string(what) + ": contiguous int32 [" + std::to_string(n) + (m ? ", " + std::to_string(m) : "") + "], got " +
        c10::toString(t->scalar_type()) + " " + shape_of(*t));
  return t->const_data_ptr<int32_t>();
}
// A tensor on the current device, from the allocator directly: at::empty's
// dispatch costs 0.45 us more, of the 5 of a call that makes two.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_generic(shape, c10::GetAllocator(at::kCUDA), c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                   std::nullopt);
}
// A buffer that a call addresses by the byte: nothing but a dense one has the
// memory that its size says (a broadcast one has less).
void dense(const char* what, const at::Tensor* t) {
  if (t && !t->is_contiguous()) bad(std::string(what) + ": not contiguous");
}
// The cache's storage, which is checked when the handle is made but may have been replaced or resized since.
void storage(const char* what, const at::Tensor* t, const af_cache_config* c) {
  dense(what, t);
  if (t->nbytes() < p_bytes(c))
    bad(std::string(what) + ": the cache needs " + std::to_string(p_bytes(c)) + " bytes, its storage has " + std::to_string(t->nbytes()));
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
bool good_type(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
af_dtype dtype_of(at::ScalarType t) { return t == at::kFloat ? AF_FP32 : AF_BF16; }

long number(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailed{};
  return v;
}
template <typename T> T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw PyFailed{};
  return static_cast<T*>(p);
}
PyObject* status(af_status s) { return PyLong_FromLong((long)s); }

void need(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) bad("wrong number of arguments");
}
void loaded() {
  if (!p_qk) throw std::runtime_error("the library is not loaded");
}

// No C++ exception leaves a function of the module.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const PyFailed&) {
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* load(PyObject* const* a, Py_ssize_t n) {
  need(n, 1);
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) throw PyFailed{};
  void* h = dlopen(path, RTLD_NOW);
  if (!h) throw std::runtime_error(dlerror());
  auto sym = [&](const char* name) {
    void* p = dlsym(h, name);
    if (!p) throw std::runtime_error(std::string("missing symbol ") + name);
    return p;
  };
  p_write = (decltype(p_write))sym("af_cache_write");
  p_read = (decltype(p_read))sym("af_cache_read");
  p_attn = (decltype(p_attn))sym("af_cache_attention");
  p_ws = (decltype(p_ws))sym("af_cache_attention_workspace_bytes");
  p_bytes = (decltype(p_bytes))sym("af_cache_bytes");
  p_qk = (decltype(p_qk))sym("af_qk_norm_rope");
  Py_RETURN_NONE;
}

// (rope address, q, k, pos, q_gain, k_gain, q_out, k_out) -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  need(n, 8);
  loaded();
  const char* what = "af_qk_norm_rope";
  const af_rope* rope = address<const af_rope>(a[0]);
  const at::Tensor *q = tensor(what, a[1], true), *k = tensor(what, a[2], true), *pos = tensor(what, a[3], false),
                   *qg = tensor(what, a[4], true), *kg = tensor(what, a[5], true), *qo = tensor(what, a[6], true),
                   *ko = tensor(what, a[7], true);
  const at::Tensor* first = q ? q : k;
  if (!first || !good_type(first->scalar_type()) || first->dim() != 3 || (k && k->dim() != 3))
    bad("af_qk_norm_rope: q or k, bf16 or fp32 [rows, heads, head_dim]");
  const int dev = c10::cuda::current_device();
  for (const at::Tensor* t : {q, k, pos, qg, kg, qo, ko}) on_device(what, t, dev);
  const at::ScalarType type = first->scalar_type();
  const int64_t rows = first->size(0), D = rope->head_dim;
  const int32_t* p = ints("af_qk_norm_rope: pos", pos, rows, 3);
  for (const at::Tensor* g : {qg, kg})
    if (g && (g->scalar_type() != at::kFloat || g->dim() != 1 || g->size(0) != D || !g->is_contiguous()))
      bad("af_qk_norm_rope: a gain is contiguous float32 [" + std::to_string(D) + "]");
  int64_t h[2] = {0, 0}, s[2] = {0, 0}, os[2] = {0, 0};
  at::Tensor made[2];
  const at::Tensor* in[2] = {q, k};
  const at::Tensor* out[2] = {q ? qo : nullptr, k ? ko : nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    h[i] = in[i]->size(1);
    s[i] = row_stride(i ? "af_qk_norm_rope: k" : "af_qk_norm_rope: q", *in[i], h[i], D, type);
    if (!out[i]) {
      made[i] = fresh({rows, h[i], D}, type);
      out[i] = &made[i];
    }
    os[i] = row_stride(i ? "af_qk_norm_rope: k_out" : "af_qk_norm_rope: q_out", *out[i], h[i], D, type);
    if (in[i]->size(0) != rows || out[i]->dim() != 3 || out[i]->size(0) != rows)
      bad("af_qk_norm_rope: q, k and the outputs have one number of rows");
  }
  if (rows > INT_MAX || h[0] > INT_MAX || h[1] > INT_MAX) bad("af_qk_norm_rope: too many rows or heads");
  auto at_ = [](const at::Tensor* t) { return t ? t->data_ptr() : nullptr; };
  const af_status st = p_qk(rope, dtype_of(type), (int)rows, at_(q), s[0], (int)h[0], at_(k), s[1], (int)h[1],
                            static_cast<const float*>(at_(qg)), static_cast<const float*>(at_(kg)), p, at_(out[0]), os[0],
                            at_(out[1]), os[1], stream_of(dev));
  if (st) return status(st);
  written(q ? qo : nullptr);
  written(k ? ko : nullptr);
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  for (int i = 0; i < 2; ++i) {
    PyObject* o = a[6 + i];
    if (made[i].defined()) {
      o = THPVariable_Wrap(made[i]);
      if (!o) {
        Py_DECREF(r);
        throw PyFailed{};
      }
    } else {
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// (config address, storage, k, v, start, count) -> None
PyObject* cache_write(PyObject* const* a, Py_ssize_t n) {
  need(n, 6);
  loaded();
  const char* what = "af_cache_write";
  const af_cache_config* c = address<const af_cache_config>(a[0]);
  const at::Tensor *store = tensor(what, a[1], false), *k = tensor(what, a[2], false), *v = tensor(what, a[3], false),
                   *start = tensor(what, a[4], true), *count = tensor(what, a[5], true);
  storage("af_cache_write: storage", store, c);
  if (k->dim() != 4 || v->sizes() != k->sizes() || k->size(0) != c->batch)
    bad("af_cache_write: k and v are [" + std::to_string(c->batch) + ", rows, " + std::to_string(c->kv_heads) + ", " +
        std::to_string(c->head_dim) + "], got " + shape_of(*k) + " and " + shape_of(*v));
  const int dev = c10::cuda::current_device();
  for (const at::Tensor* t : {store, k, v, start, count}) on_device(what, t, dev);
  const int32_t *s = ints("af_cache_write: start", start, c->batch), *m = ints("af_cache_write: count", count, c->batch);
  const int64_t ks = row_stride("af_cache_write: k", *k, c->kv_heads, c->head_dim, at::kBFloat16),
                vs = row_stride("af_cache_write: v", *v, c->kv_heads, c->head_dim, at::kBFloat16);
  if (k->size(1) > INT_MAX) bad("af_cache_write: too many rows");
  const af_status st = p_write(c, store->data_ptr(), (int)k->size(1), k->data_ptr(), batch_stride(*k, ks), ks,
                               v->data_ptr(), batch_stride(*v, vs), vs, s, m, stream_of(dev));
  if (st) return status(st);
  written(store);
  Py_RETURN_NONE;
}

// (config address, storage, rows, start, count, fp32, k, v) -> (k, v)
PyObject* cache_read(PyObject* const* a, Py_ssize_t n) {
  need(n, 8);
  loaded();
  const char* what = "af_cache_read";
  const af_cache_config* c = address<const af_cache_config>(a[0]);
  const at::Tensor *store = tensor(what, a[1], false), *start = tensor(what, a[3], true), *count = tensor(what, a[4], true),
                   *k = tensor(what, a[6], true), *v = tensor(what, a[7], true);
  const long rows = number(a[2]);
  const at::ScalarType type = number(a[5]) ? at::kFloat : at::kBFloat16;
  if (rows < 0 || rows > INT_MAX || !k != !v) bad("af_cache_read: rows >= 0, and k and v both given or neither");
  storage("af_cache_read: storage", store, c);
  const int dev = c10::cuda::current_device();
  at::Tensor made[2];
  if (!k) {
    for (at::Tensor& t : made) t = fresh({c->batch, rows, c->kv_heads, c->head_dim}, type);
    k = &made[0];
    v = &made[1];
  }
  for (const at::Tensor* t : {store, k, v, start, count}) on_device(what, t, dev);
  const int32_t *s = ints("af_cache_read: start", start, c->batch), *m = ints("af_cache_read: count", count, c->batch);
  auto unlike = [&] {
    bad("af_cache_read: k and v are [" + std::to_string(c->batch) + ", " + std::to_string(rows) + ", " +
        std::to_string(c->kv_heads) + ", " + std::to_string(c->head_dim) + "] of one layout");
  };
  if (k->dim() != 4 || k->size(0) != c->batch || k->size(1) != rows || v->sizes() != k->sizes()) unlike();
  const int64_t ks = row_stride("af_cache_read: k", *k, c->kv_heads, c->head_dim, type);
  // (strides of dimensions of one element say nothing)
  const int64_t vs = row_stride("af_cache_read: v", *v, c->kv_heads, c->head_dim, type);
  if (vs != ks || batch_stride(*v, vs) != batch_stride(*k, ks)) unlike();
  const af_status st = p_read(c, store->data_ptr(), (int)rows, s, m, dtype_of(type), k->data_ptr(), v->data_ptr(),
                              batch_stride(*k, ks), ks, stream_of(dev));
  if (st) return status(st);
  if (!made[0].defined()) {
    written(k);
    written(v);
  }
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyFailed{};
  for (int i = 0; i < 2; ++i) {
    PyObject* o = a[6 + i];
    if (made[i].defined()) {
      o = THPVariable_Wrap(made[i]);
      if (!o) {
        Py_DECREF(r);
        throw PyFailed{};
      }
    } else {
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// (config address, storage, q, length, n_q, causal, scale, ws, out) -> out
PyObject* cache_attention(PyObject* const* a, Py_ssize_t n) {
  need(n, 9);
  loaded();
  const char* what = "af_cache_attention";
  const af_cache_config* c = address<const af_cache_config>(a[0]);
  const at::Tensor *store = tensor(what, a[1], false), *q = tensor(what, a[2], false), *length = tensor(what, a[3], false),
                   *nq = tensor(what, a[4], true), *ws = tensor(what, a[7], true), *out = tensor(what, a[8], true);
  storage("af_cache_attention: storage", store, c);
  dense("af_cache_attention: ws", ws);
  if (q->dim() != 4 || q->size(0) != c->batch)
    bad("af_cache_attention: q is [" + std::to_string(c->batch) + ", rows, heads, " + std::to_string(c->head_dim) +
        "], got " + shape_of(*q));
  const double scale = PyFloat_AsDouble(a[6]);
  if (scale == -1.0 && PyErr_Occurred()) throw PyFailed{};
  const long causal = number(a[5]);
  const int64_t rows = q->size(1), heads = q->size(2);
  if (rows > INT_MAX || heads > INT_MAX) bad("af_cache_attention: too many rows or heads");
  const int dev = c10::cuda::current_device();
  for (const at::Tensor* t : {store, q, length, nq, ws, out}) on_device(what, t, dev);
  const int32_t *len = ints("af_cache_attention: length", length, c->batch), *m = ints("af_cache_attention: n_q", nq, c->batch);
  const int64_t qs = row_stride("af_cache_attention: q", *q, heads, c->head_dim, at::kBFloat16);
  at::Tensor made, work;
  if (!out) {
    made = fresh(q->sizes(), at::kBFloat16);
    out = &made;
  }
  if (out->sizes() != q->sizes()) bad("af_cache_attention: out is " + shape_of(*q) + ", got " + shape_of(*out));
  const int64_t os = row_stride("af_cache_attention: out", *out, heads, c->head_dim, at::kBFloat16);
  if (!ws) {
    const size_t bytes = p_ws(c, (int)heads, (int)rows);
    work = fresh({(int64_t)(bytes < 256 ? 256 : bytes)}, at::kByte);
    ws = &work;
  }
  const af_status st = p_attn(c, store->data_ptr(), (int)rows, (int)heads, q->data_ptr(), batch_stride(*q, qs), qs, len, m,
                              causal != 0, (float)scale, out->data_ptr(), batch_stride(*out, os), os, ws->data_ptr(),
                              (size_t)ws->nbytes(), stream_of(dev));
  if (st) return status(st);
  if (!made.defined()) written(out);
  if (made.defined()) {
    PyObject* o = THPVariable_Wrap(made);
    if (!o) throw PyFailed{};
    return o;
  }
  Py_INCREF(a[8]);
  return a[8];
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f>)), METH_FASTCALL
PyMethodDef methods[] = {{"load", FAST(load), "resolves the library's calls"},
                         {"qk_norm_rope", FAST(qk_norm_rope), nullptr},
                         {"cache_write", FAST(cache_write), nullptr},
                         {"cache_read", FAST(cache_read), nullptr},
                         {"cache_attention", FAST(cache_attention), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__binding(void) { return PyModule_Create(&module); }
