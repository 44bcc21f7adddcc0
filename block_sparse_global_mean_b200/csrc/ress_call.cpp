// The binding's common case in C++: calls of the cross-attention and cache
// operators with nothing but their inputs, on the current device and stream.
// Small calls take a few microseconds on the GPU, less than a dozen attribute
// lookups and three allocations take in Python (a plan: 15.6 us a call through
// ctypes, 5.4 us from here).  Each function checks what the Python binding checks and
// returns None where anything is not as it should be, or not common (another
// device, tensor subclasses, an error from the library): the Python code then
// does the call, or says what is wrong with it.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <string.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ress.h"

namespace {

decltype(&ress_cross_workspace_bytes) cross_bytes;
decltype(&ress_cross_bwd_workspace_bytes) cross_bwd_bytes;
decltype(&ress_cross_attn) cross_attn;
decltype(&ress_cross_attn_bwd) cross_attn_bwd;
decltype(&ress_cache_plan) cache_plan;
decltype(&ress_cache_append) cache_append;
decltype(&ress_cache_attn_workspace_bytes) cache_attn_bytes;
decltype(&ress_cache_attn) cache_attn;

template <typename F>
bool find(void* lib, const char* name, F* f) {
  *f = reinterpret_cast<F>(dlsym(lib, name));
  return *f != nullptr;
}

// init(path of the library, which is loaded already, and the tag of this torch and
// Python: another one's objects would be read by the layouts compiled in here)
PyObject* init(PyObject*, PyObject* args) {
  const char *p, *tag;
  if (!PyArg_ParseTuple(args, "ss", &p, &tag)) return nullptr;
  if (strcmp(tag, RESS_CALL_TAG) != 0) {
    PyErr_Format(PyExc_ImportError, "built for %s, not for %s", RESS_CALL_TAG, tag);
    return nullptr;
  }
  void* lib = dlopen(p, RTLD_NOW);
  if (lib == nullptr || !find(lib, "ress_cross_workspace_bytes", &cross_bytes) ||
      !find(lib, "ress_cross_bwd_workspace_bytes", &cross_bwd_bytes) ||
      !find(lib, "ress_cross_attn", &cross_attn) ||
      !find(lib, "ress_cross_attn_bwd", &cross_attn_bwd) ||
      !find(lib, "ress_cache_plan", &cache_plan) ||
      !find(lib, "ress_cache_append", &cache_append) ||
      !find(lib, "ress_cache_attn_workspace_bytes", &cache_attn_bytes) ||
      !find(lib, "ress_cache_attn", &cache_attn)) {
    PyErr_Format(PyExc_ImportError, "%s: %s", p, dlerror());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// The arguments of a call; ok turns false at the first that is not common.
struct Call {
  PyObject* const* args;
  bool ok = true;
  int device = -1;

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : args(a), ok(n == want) {}

  // A CUDA tensor on the current device.
  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_CheckExact(args[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (device < 0) {
      device = c10::cuda::current_device();
    }
    if (t.get_device() != device) return fail();
    return &t;
  }
  // A dense one of a given type and shape (-1: any).
  void* dense(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->dim() != (int64_t)shape.size() || !t->is_contiguous())
      return fail<void>();
    int64_t d = 0;
    for (int64_t n : shape) {
      if (n >= 0 && t->size(d) != n) return fail<void>();
      ++d;
    }
    return t->data_ptr();
  }
  void* dense_or_none(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return ok && args[i] == Py_None ? nullptr : dense(i, type, shape);
  }
  // Token rows [n, heads, d] whose heads stand together; the elements between
  // them, 0 if dense.
  const at::Tensor* rows(int i, int64_t* stride) {
    const at::Tensor* t = tensor(i);
    if (t == nullptr || t->dim() != 3) return fail();
    *stride = 0;
    if (t->is_contiguous()) return t;
    if (t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != t->size(2)) ||
        t->stride(0) < t->size(1) * t->size(2))
      return fail();
    *stride = t->stride(0);
    return t;
  }
  long long number(int i) {
    if (!ok) return 0;
    const long long x = PyLong_Check(args[i]) ? PyLong_AsLongLong(args[i]) : -1;
    if (x < 0 || x > 0x7fffffff) {
      PyErr_Clear();
      ok = false;
      return 0;
    }
    return x;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }

  template <typename T = const at::Tensor>
  T* fail() {
    ok = false;
    return nullptr;
  }
};

int32_t dtype_of(const at::Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? RESS_BF16 : t.scalar_type() == at::kFloat ? RESS_F32 : -1;
}

at::Tensor workspace(size_t need, const at::Tensor& like) {
  return at::empty({(int64_t)need}, like.options().dtype(at::kByte));
}

// Entries [at, at + n) of a new tensor without a gradient, as a tensor of their own
// on its storage (a view by the dispatcher takes 0.6 us).
at::Tensor part(const at::Tensor& all, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                          all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// Shape and arrays of a packed batch: arguments 0..6 are q, k, v, q_offsets,
// kv_offsets, q_lens, kv_lens.
struct Cross {
  const at::Tensor *q, *k, *v;
  ress_cross_shape shape{};
  const int32_t *qo = nullptr, *ko = nullptr, *ql = nullptr, *kl = nullptr;

  explicit Cross(Call& c) {
    q = c.rows(0, &shape.q_stride);
    k = c.rows(1, &shape.k_stride);
    v = c.rows(2, &shape.v_stride);
    if (!c.ok) return;
    if (q->scalar_type() != at::kBFloat16 || k->scalar_type() != at::kBFloat16 ||
        v->scalar_type() != at::kBFloat16 || v->sizes() != k->sizes() || k->size(2) != q->size(2) ||
        (c.args[3] == Py_None) != (c.args[4] == Py_None)) {
      c.ok = false;
      return;
    }
    int64_t seqs = 1;
    if (c.args[3] != Py_None) {
      const at::Tensor* t = c.tensor(3);
      if (!c.ok || t->dim() != 1 || t->size(0) < 2) {
        c.ok = false;
        return;
      }
      seqs = t->size(0) - 1;
      qo = static_cast<int32_t*>(c.dense(3, at::kInt, {seqs + 1}));
      ko = static_cast<int32_t*>(c.dense(4, at::kInt, {seqs + 1}));
    }
    ql = static_cast<int32_t*>(c.dense_or_none(5, at::kInt, {seqs}));
    kl = static_cast<int32_t*>(c.dense_or_none(6, at::kInt, {seqs}));
    if (q->size(1) > 64 || k->size(1) > 64 || seqs > 8192) c.ok = false;   // (fits 32 bits)
    shape.nq = q->size(0);
    shape.nk = k->size(0);
    shape.seqs = (int32_t)seqs;
    shape.heads = (int32_t)q->size(1);
    shape.kv_heads = (int32_t)k->size(1);
    shape.head_dim = (int32_t)q->size(2);
    shape.dtype = RESS_BF16;
  }
};

// Parts of a cache: arguments i .. i + 3 are k, v, k_scale, v_scale.
struct Cache {
  void *k, *v;
  float *ks, *vs;
  ress_cache_shape shape{};

  Cache(Call& c, int i) {
    const at::Tensor* t = c.tensor(i);
    if (!c.ok || t->dim() != 4 || t->size(0) > 0x7fffffff || t->size(1) > 64 || t->size(2) > 128) {
      c.ok = false;
      return;
    }
    const int64_t pages = t->size(0), heads = t->size(1), page = t->size(2), d = t->size(3);
    k = c.dense(i, at::kFloat8_e4m3fn, {pages, heads, page, d});
    v = c.dense(i + 1, at::kFloat8_e4m3fn, {pages, heads, page, d});
    ks = static_cast<float*>(c.dense(i + 2, at::kFloat, {pages, heads}));
    vs = static_cast<float*>(c.dense(i + 3, at::kFloat, {pages, heads}));
    shape = {(int32_t)pages, (int32_t)page, (int32_t)heads, (int32_t)d, 1, 1};
  }
};

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined()) o = THPVariable_Wrap(t);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No C++ exception passes into the interpreter: the Python code makes the call
// again and raises what there is to raise.
template <typename F>
PyObject* guarded(F f) {
  try {
    if (PyObject* r = f()) return r;
  } catch (...) {
  }
  Py_RETURN_NONE;
}

// cross_attn(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens, want_lse) -> (out, lse)
PyObject* py_cross_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 8);
    if (!c.ok) return nullptr;
    Cross x(c);
    if (!c.ok) return nullptr;
    const at::Tensor out = at::empty(x.q->sizes(), x.q->options());
    at::Tensor lse;
    if (args[7] == Py_True)
      lse = at::empty({x.q->size(1), x.q->size(0)}, x.q->options().dtype(at::kFloat));
    const size_t need = cross_bytes(&x.shape);
    const at::Tensor ws = workspace(need, *x.q);
    if (cross_attn(&x.shape, x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), x.qo, x.ko, x.ql,
                   x.kl, out.data_ptr(), lse.defined() ? lse.data_ptr<float>() : nullptr,
                   ws.data_ptr(), need, c.stream()) != RESS_OK)
      return nullptr;
    return pack({out, lse});
  });
}

// cross_attn_bwd(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens, out, lse, dout) -> (dq, dk, dv)
PyObject* py_cross_attn_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 10);
    if (!c.ok) return nullptr;
    Cross x(c);
    if (!c.ok) return nullptr;
    const int64_t nq = x.q->size(0), h = x.q->size(1), d = x.q->size(2);
    const void* out = c.dense(7, at::kBFloat16, {nq, h, d});
    const float* lse = static_cast<float*>(c.dense(8, at::kFloat, {h, nq}));
    const void* dout = c.dense(9, at::kBFloat16, {nq, h, d});
    if (!c.ok) return nullptr;
    const at::Tensor dq = at::empty(x.q->sizes(), x.q->options());
    const at::Tensor dk = at::empty(x.k->sizes(), x.k->options());
    const at::Tensor dv = at::empty(x.k->sizes(), x.k->options());
    const size_t need = cross_bwd_bytes(&x.shape);
    const at::Tensor ws = workspace(need, *x.q);
    if (cross_attn_bwd(&x.shape, x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), out, lse, dout,
                       x.qo, x.ko, x.ql, x.kl, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                       ws.data_ptr(), need, c.stream()) != RESS_OK)
      return nullptr;
    return pack({dq, dk, dv});
  });
}

// cache_plan(added, lengths, table, free_pages, cursor, page, tokens, pages or None)
//   -> (offsets, slots, new_lengths, new_cursor)
PyObject* py_cache_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 8);
    const at::Tensor* added = c.tensor(0);
    const at::Tensor* table = c.tensor(2);
    const at::Tensor* free_pages = c.tensor(3);
    if (!c.ok || table->dim() != 2 || free_pages->dim() != 1) return nullptr;
    const int64_t r = table->size(0), width = table->size(1), n_free = free_pages->size(0);
    const int32_t* a = static_cast<int32_t*>(c.dense(0, at::kInt, {r}));
    const int32_t* l = static_cast<int32_t*>(c.dense(1, at::kInt, {r}));
    int32_t* t = static_cast<int32_t*>(c.dense(2, at::kInt, {r, width}));
    const int32_t* f = static_cast<int32_t*>(c.dense(3, at::kInt, {n_free}));
    const int32_t* cursor = static_cast<int32_t*>(c.dense(4, at::kInt, {1}));
    const long long page = c.number(5), tokens = c.number(6);
    const long long pages = c.ok && args[7] != Py_None ? c.number(7)
                            : page > 0                 ? 0x7fffffff / page
                                                       : 0;
    if (!c.ok || r > 8192 || width > 0x7fffffff || n_free > 0x7fffffff) return nullptr;
    const ress_cache_shape shape{(int32_t)pages, (int32_t)page, 1, 64, (int32_t)r, (int32_t)width};
    const at::Tensor all = at::empty({r + 1 + tokens + r + 1}, added->options());
    const at::Tensor made[4] = {part(all, 0, r + 1), part(all, r + 1, tokens),
                                part(all, r + 1 + tokens, r), part(all, 2 * r + 1 + tokens, 1)};
    int32_t* p = all.data_ptr<int32_t>();
    if (cache_plan(&shape, a, l, t, f, (int32_t)n_free, cursor, (int32_t)tokens, p, p + r + 1,
                   p + r + 1 + tokens, p + 2 * r + 1 + tokens, c.stream()) != RESS_OK)
      return nullptr;
    return pack({made[0], made[1], made[2], made[3]});
  });
}

// cache_append(k, v, slots, cache.k, cache.v, cache.k_scale, cache.v_scale) -> True
PyObject* py_cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 7);
    int64_t ks = 0, vs = 0;
    const at::Tensor* k = c.rows(0, &ks);
    const at::Tensor* v = c.rows(1, &vs);
    if (!c.ok) return nullptr;
    Cache x(c, 3);
    const int64_t tokens = k->size(0);
    const int32_t* slots = static_cast<int32_t*>(c.dense(2, at::kInt, {tokens}));
    const int32_t dtype = dtype_of(*k);
    if (!c.ok || dtype < 0 || v->scalar_type() != k->scalar_type() || v->sizes() != k->sizes() ||
        k->size(1) != x.shape.kv_heads || k->size(2) != x.shape.head_dim || tokens > 0x7fffffff)
      return nullptr;
    if (cache_append(&x.shape, k->data_ptr(), v->data_ptr(), dtype, ks, vs, slots, (int32_t)tokens,
                     x.k, x.v, x.ks, x.vs, c.stream()) != RESS_OK)
      return nullptr;
    Py_RETURN_TRUE;
  });
}

// cache_attn(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, offsets, step,
//            want_lse) -> (out, lse)
PyObject* py_cache_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 10);
    int64_t stride = 0;
    const at::Tensor* q = c.rows(0, &stride);
    if (!c.ok) return nullptr;
    Cache x(c, 1);
    const at::Tensor* table = c.tensor(5);
    if (!c.ok || table->dim() != 2) return nullptr;
    const int64_t r = table->size(0), width = table->size(1), tokens = q->size(0);
    const int32_t* t = static_cast<int32_t*>(c.dense(5, at::kInt, {r, width}));
    const int32_t* lengths = static_cast<int32_t*>(c.dense(6, at::kInt, {r}));
    const int32_t* offsets = static_cast<int32_t*>(c.dense(7, at::kInt, {r + 1}));
    const long long step = c.number(8);
    if (!c.ok || q->scalar_type() != at::kBFloat16 || q->size(2) != x.shape.head_dim ||
        q->size(1) > 64 || r > 8192 || width > 0x7fffffff || tokens > 0x7fffffff)
      return nullptr;
    x.shape.requests = (int32_t)r;
    x.shape.max_pages = (int32_t)width;
    const int32_t heads = (int32_t)q->size(1);
    const at::Tensor out = at::empty(q->sizes(), q->options());
    at::Tensor lse;
    if (args[9] == Py_True) lse = at::empty({q->size(1), tokens}, q->options().dtype(at::kFloat));
    const size_t need = cache_attn_bytes(&x.shape, heads, (int32_t)tokens);
    const at::Tensor ws = workspace(need, *q);
    if (cache_attn(&x.shape, heads, (int32_t)tokens, q->data_ptr(), stride, x.k, x.v, x.ks, x.vs, t,
                   lengths, offsets, (int32_t)step, out.data_ptr(),
                   lse.defined() ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), need,
                   c.stream()) != RESS_OK)
      return nullptr;
    return pack({out, lse});
  });
}

template <typename F>
constexpr PyCFunction as_c(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"cross_attn", as_c(py_cross_attn), METH_FASTCALL, nullptr},
    {"cross_attn_bwd", as_c(py_cross_attn_bwd), METH_FASTCALL, nullptr},
    {"cache_plan", as_c(py_cache_plan), METH_FASTCALL, nullptr},
    {"cache_append", as_c(py_cache_append), METH_FASTCALL, nullptr},
    {"cache_attn", as_c(py_cache_attn), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ress_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ress_call() { return PyModule_Create(&module); }
