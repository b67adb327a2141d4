// Fast path of the Python binding for the calls of a speculative step: reads
// the tensors' shapes, types, strides and addresses and makes the C call.  Each
// function returns the mla_status, or None where an argument is not what the
// call takes, which Python then explains.  (A small call's kernels take 2 to 4
// us; the same tests and the call through ctypes take 10, here 2 to 4.)
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "mla_pages.h"
#include "mla_rope.h"
#include "mla_tree.h"
#include "mla_verify.h"

namespace {

using at::ScalarType;

// The arguments of a call; `ok` is false once one of them does not fit.
struct Call {
  PyObject* const* args;
  bool ok = true;
  int dev = -1;

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : args(a), ok(n == want) {}

  // A dense CUDA tensor; all of a call's are on one device.
  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_Check(args[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (dev < 0) dev = t.get_device();
    if (t.get_device() != dev) return fail();
    return &t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  bool none(int i) const { return args[i] == Py_None; }

  // A contiguous tensor of the given type and shape.
  void* full(int i, ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || t->dim() != static_cast<int64_t>(shape.size()) || !t->is_contiguous())
      return fail(), nullptr;
    int64_t k = 0;
    for (const int64_t n : shape)
      if (t->size(k++) != n) return fail(), nullptr;
    return t->data_ptr();
  }
  template <typename T>
  T* vec(int i, ScalarType type, int64_t n) {
    return static_cast<T*>(full(i, type, {n}));
  }
  int32_t* ints(int i, int64_t n) { return vec<int32_t>(i, ScalarType::Int, n); }
  float* floats(int i, int64_t n) { return vec<float>(i, ScalarType::Float, n); }

  // A one-dimensional tensor's length.
  int64_t length(int i) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != 1) return fail(), 0;
    return t->size(0);
  }
  // int32 [rows, any] with unit column stride.
  int32_t* table(int i, int64_t rows, int64_t* cols, int64_t* stride) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != ScalarType::Int || t->dim() != 2 || t->size(0) != rows || t->stride(1) != 1 ||
        t->stride(0) < t->size(1))
      return fail(), nullptr;
    *cols = t->size(1);
    *stride = t->stride(0);
    return static_cast<int32_t*>(t->data_ptr());
  }
  int32_t* status(int i) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != ScalarType::Int || t->numel() < 1) return fail(), nullptr;
    return static_cast<int32_t*>(t->data_ptr());
  }
  void* workspace(int i, size_t* bytes) {
    const at::Tensor* t = tensor(i);
    if (!t || !t->is_contiguous()) return fail(), nullptr;
    *bytes = t->nbytes();
    return t->data_ptr();
  }
  static int dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
      case ScalarType::BFloat16: return MLA_KV_BF16;
      case ScalarType::Byte:
      case ScalarType::Float8_e4m3fn: return MLA_KV_FP8_E4M3;
      default: return -1;
    }
  }
  // A cache [num_pages, 64, 576], or one per layer with contiguous layers.
  struct Cache {
    void* at = nullptr;
    int64_t layers = 1, pages = 0, page_size = 0, step = 0;
    int dtype = 0;
  };
  Cache cache(int i, bool many) {
    Cache c;
    const at::Tensor* t = tensor(i);
    if (!t || dtype_of(*t) < 0) return fail(), c;
    const int64_t d = t->dim();
    if (d != 3 && !(many && d == 4)) return fail(), c;
    if (t->size(d - 1) != 576 || t->stride(d - 1) != 1 || t->stride(d - 2) != 576 ||
        (t->size(d - 3) > 1 && t->stride(d - 3) != t->size(d - 2) * 576))
      return fail(), c;
    c.at = t->data_ptr();
    c.pages = t->size(d - 3);
    c.page_size = t->size(d - 2);
    c.dtype = dtype_of(*t);
    if (d == 4) {
      c.layers = t->size(0);
      c.step = c.layers > 1 ? t->stride(0) * static_cast<int64_t>(t->element_size()) : 0;
    }
    return c;
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  int32_t i32(int64_t v) {
    if (v < INT_MIN || v > INT_MAX) ok = false;
    return static_cast<int32_t>(v);
  }
  // The stream given, or the device's current one; the device has to be the current one.
  void* stream(int i) {
    if (!ok || c10::cuda::current_device() != dev) return fail(), nullptr;
    if (none(i)) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    PyObject* h = PyObject_GetAttrString(args[i], "cuda_stream");
    void* s = h ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return fail(), nullptr;
    }
    return s;
  }
};

// The C call, with the interpreter's lock given up meanwhile: a launch waits
// where the stream's queue is full, and what it waits for may need the lock (a
// callback, another thread).  The caller's arguments keep the tensors alive.
template <typename F>
int unlocked(F call) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return call();
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {  // what went wrong is found again, and explained, in Python
    Py_RETURN_NONE;
  }
}

// q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, scale, kv_scale, out, lse, workspace, stream
PyObject* decode_tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 13);
    const at::Tensor* q = c.tensor(0);
    if (!q || q->dim() != 3) Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), B = c.length(4);
    int64_t cols = 0, stride = 0;
    size_t bytes = 0;
    const auto bf16 = ScalarType::BFloat16;
    void* qn = c.full(0, bf16, {T, H, 512});
    void* qp = c.full(1, bf16, {T, H, 64});
    const Call::Cache kv = c.cache(2, false);
    int32_t* table = c.table(3, B, &cols, &stride);
    int32_t* lens = c.ints(4, B);
    int32_t* cu = c.ints(5, B + 1);
    int32_t* parents = c.ints(6, T);
    const float scale = c.number(7), kv_scale = c.number(8);
    void* out = c.full(9, bf16, {T, H, 512});
    float* lse = static_cast<float*>(c.full(10, ScalarType::Float, {T, H}));
    void* ws = c.workspace(11, &bytes);
    void* s = c.stream(12);
    const mla_prefill_dims d = {c.i32(B),    c.i32(H),      c.i32(T),      c.i32(kv.page_size), c.i32(kv.pages),
                                c.i32(cols), c.i32(stride), kv.dtype};
    if (!c.ok) Py_RETURN_NONE;
    return PyLong_FromLong(unlocked([&] {
      return mla_decode_tree(&d, qn, qp, kv.at, table, lens, cu, parents, scale, kv_scale, out, lse, ws, bytes, s);
    }));
  });
}

// kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, new_lens, status, stream
PyObject* tree_commit(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 9);
    const Call::Cache kv = c.cache(0, true);
    const at::Tensor* p = c.tensor(4);
    if (!p || p->dim() != 2 || kv.page_size != 64) Py_RETURN_NONE;
    const int64_t B = c.length(2), path_cols = p->size(1);
    int64_t cols = 0, stride = 0;
    int32_t* table = c.table(1, B, &cols, &stride);
    int32_t* lens = c.ints(2, B);
    int32_t* cu = c.ints(3, B + 1);
    int32_t* path = static_cast<int32_t*>(c.full(4, ScalarType::Int, {B, path_cols}));
    int32_t* num = c.ints(5, B);
    int32_t* new_lens = c.ints(6, B);
    int32_t* status = c.status(7);
    void* s = c.stream(8);
    const mla_tree_commit_dims d = {c.i32(B),    c.i32(kv.layers), c.i32(path_cols), c.i32(kv.pages),
                                    c.i32(cols), c.i32(stride),    kv.dtype,         0,
                                    kv.step};
    if (!c.ok) Py_RETURN_NONE;
    return PyLong_FromLong(
        unlocked([&] { return mla_tree_commit(&d, kv.at, table, lens, cu, path, num, new_lens, status, s); }));
  });
}

// target, draft, tokens, parents, cu_q_lens, accept, sample, path, tokens_out, num_out, status, stream
PyObject* verify(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 12);
    const at::Tensor* t = c.tensor(0);
    const at::Tensor* p = c.tensor(7);
    if (!t || !p || t->dim() != 2 || p->dim() != 2) Py_RETURN_NONE;
    const int64_t T = t->size(0), V = t->size(1), B = c.length(6), cols = p->size(1);
    auto rows = [&](int i, int64_t* stride) -> const float* {
      const at::Tensor* x = c.tensor(i);
      if (!x || x->scalar_type() != ScalarType::Float || x->dim() != 2 || x->size(0) != T || x->size(1) != V ||
          x->stride(1) != 1 || (T > 1 && x->stride(0) < V)) {
        c.ok = false;
        return nullptr;
      }
      *stride = T > 1 ? x->stride(0) : V;
      return static_cast<const float*>(x->data_ptr());
    };
    int64_t ts = 0, ds = 0;
    const float* target = rows(0, &ts);
    const float* draft = c.none(1) ? nullptr : rows(1, &ds);
    int32_t* tokens = c.ints(2, T);
    int32_t* parents = c.ints(3, T);
    int32_t* cu = c.ints(4, B + 1);
    float* accept = c.floats(5, T);
    float* sample = c.floats(6, B);
    int32_t* path = static_cast<int32_t*>(c.full(7, ScalarType::Int, {B, cols}));
    int32_t* out = static_cast<int32_t*>(c.full(8, ScalarType::Int, {B, cols}));
    int32_t* num = c.ints(9, B);
    int32_t* status = c.status(10);
    void* s = c.stream(11);
    const mla_verify_dims d = {c.i32(B), c.i32(T), c.i32(V), c.i32(cols), ts, ds};
    if (!c.ok) Py_RETURN_NONE;
    return PyLong_FromLong(unlocked([&] {
      return mla_verify(&d, target, draft, tokens, parents, cu, accept, sample, path, out, num, status, s);
    }));
  });
}

// new_lens, page_table, page_refs, page_table_out, page_refs_out, workspace, stream
PyObject* page_resize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 7);
    const int64_t B = c.length(0), P = c.length(2);
    int64_t cols = 0, stride = 0, out_cols = 0, out_stride = 0;
    size_t bytes = 0;
    int32_t* lens = c.ints(0, B);
    int32_t* table = c.table(1, B, &cols, &stride);
    int32_t* refs = c.ints(2, P);
    int32_t* table_out = c.table(3, B, &out_cols, &out_stride);
    int32_t* refs_out = c.ints(4, P);
    void* ws = c.workspace(5, &bytes);
    void* s = c.stream(6);
    const mla_page_resize_dims d = {c.i32(B), c.i32(P), c.i32(cols), c.i32(stride), c.i32(out_stride)};
    if (!c.ok || cols != out_cols) Py_RETURN_NONE;
    return PyLong_FromLong(
        unlocked([&] { return mla_page_resize(&d, lens, table, refs, table_out, refs_out, ws, bytes, s); }));
  });
}

// src, seq_lens, page_table, page_refs, kv_cache, page_table_out, page_refs_out, workspace, stream
PyObject* page_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 9);
    const int64_t C = c.length(0), S = c.length(1);
    int64_t cols = 0, stride = 0, out_cols = 0, out_stride = 0;
    size_t bytes = 0;
    const Call::Cache kv = c.cache(4, true);
    int32_t* src = c.ints(0, C);
    int32_t* lens = c.ints(1, S);
    int32_t* table = c.table(2, S, &cols, &stride);
    int32_t* refs = c.ints(3, kv.pages);
    int32_t* table_out = c.table(5, C, &out_cols, &out_stride);
    int32_t* refs_out = c.ints(6, kv.pages);
    void* ws = c.workspace(7, &bytes);
    void* s = c.stream(8);
    const mla_page_fork_dims d = {c.i32(S),    c.i32(C),      c.i32(kv.layers),  c.i32(kv.pages),
                                  c.i32(cols), c.i32(stride), c.i32(out_stride), kv.dtype,
                                  kv.step};
    if (!c.ok || cols != out_cols || kv.page_size != 64) Py_RETURN_NONE;
    return PyLong_FromLong(unlocked([&] {
      return mla_page_fork(&d, src, lens, table, refs, kv.at, table_out, refs_out, ws, bytes, s);
    }));
  });
}

// plan, q_pe, rows, positions, page_table, seq_lens, cu_q_lens, kv_scale, q_out, kv_cache, status, stream
PyObject* rope_pack(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 12);
    const at::Tensor* q = c.tensor(1);
    const at::Tensor* r = c.tensor(2);
    const auto bf16 = ScalarType::BFloat16;
    if (!q || !r || q->dim() != 3 || q->size(2) != 64 || q->scalar_type() != bf16 || q->stride(2) != 1) Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), B = c.length(5);
    if (r->dim() != 2 || r->size(0) != T || r->size(1) != 576 || r->scalar_type() != bf16 || r->stride(1) != 1)
      Py_RETURN_NONE;
    int64_t cols = 0, stride = 0;
    int32_t* positions = c.none(3) ? nullptr : c.ints(3, T);
    int32_t* table = c.table(4, B, &cols, &stride);
    int32_t* lens = c.ints(5, B);
    int32_t* cu = c.ints(6, B + 1);
    const float kv_scale = c.number(7);
    const void *qp = q->data_ptr(), *rows = r->data_ptr();
    void* out = c.full(8, bf16, {T, H, 64});
    const Call::Cache kv = c.cache(9, false);
    int32_t* status = c.status(10);
    void* s = c.stream(11);
    const mla_rope_dims d = {c.i32(B),      c.i32(H), c.i32(T),     c.i32(kv.pages), c.i32(cols),
                             c.i32(stride), kv.dtype, 0,            q->stride(0),    q->stride(1),
                             r->stride(0)};
    if (!c.ok || kv.page_size != 64) Py_RETURN_NONE;
    Py_buffer plan;  // the plan's memory
    if (PyObject_GetBuffer(args[0], &plan, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    int rc = 1;
    if (plan.len == static_cast<Py_ssize_t>(sizeof(mla_rope_plan)))
      rc = unlocked([&] {
        return mla_rope_pack(&d, static_cast<const mla_rope_plan*>(plan.buf), qp, rows, positions, table, lens, cu,
                             kv_scale, out, kv.at, status, s);
      });
    PyBuffer_Release(&plan);
    if (rc == 1) Py_RETURN_NONE;
    return PyLong_FromLong(rc);
  });
}

#define FAST(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FAST(decode_tree), FAST(tree_commit), FAST(verify),  FAST(page_resize),
                         FAST(page_fork),   FAST(rope_pack),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
