// Native argument marshalling for the single-token serving calls: torch
// tensors to the pointers and sizes of include/fdllm.h. The calls take a few
// microseconds on the GPU, and checking fourteen tensors in Python took longer
// than that. No arithmetic and no launch happens here; the entry points are
// those of libfdllm.so, handed over by address (bind).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "fdllm.h"

namespace {

decltype(&fdllm_plan_step) plan_step_fn = nullptr;
decltype(&fdllm_release_blocks) release_blocks_fn = nullptr;
decltype(&fdllm_decode_workspace_bytes) workspace_fn = nullptr;
decltype(&fdllm_decode_attention) decode_fn = nullptr;
decltype(&fdllm_linear) linear_fn = nullptr;

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  TORCH_CHECK_TYPE(t, name, " must be a tensor");
  return *t;
}

// The tensors of one call lie on one device, which is made current.
struct Call {
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;

  static const at::Tensor& on_gpu(const at::Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    return t;
  }
  Call(const at::Tensor& t, const char* name) : device(on_gpu(t, name).device()), guard(device) {}

  void* stream() const {
    return reinterpret_cast<void*>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  }

  // What a call returns or works in. (Past the dispatcher: 2.6 us of checks and
  // allocations for a decode call instead of 3.5.)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
  }

  void here(const at::Tensor& t, const char* name) const {
    TORCH_CHECK_VALUE(t.device() == device, name, " must be a CUDA tensor on device ",
                      (int)device.index());
  }

  // Address of a contiguous tensor of this type and shape (null for none).
  void* arg(const at::Tensor* t, const char* name, at::ScalarType type,
            at::IntArrayRef shape) const {
    if (!t) return nullptr;
    here(*t, name);
    TORCH_CHECK_VALUE(t->scalar_type() == type, name, " must be ", type, ", got ", t->scalar_type());
    TORCH_CHECK_VALUE(t->sizes() == shape, name, " must have shape ", shape, ", got ", t->sizes());
    TORCH_CHECK_VALUE(t->is_contiguous(), name, " must be contiguous");
    return t->data_ptr();
  }

  template <typename T>
  T* i32(PyObject* o, const char* name, at::IntArrayRef shape) const {
    return static_cast<T*>(arg(tensor(o, name), name, at::kInt, shape));
  }

  // The same for a matrix whose rows are contiguous but may lie apart; the
  // stride of a single row says nothing.
  void* rows(const at::Tensor* t, const char* name, at::ScalarType type, int64_t n, int64_t width,
             int64_t& stride) const {
    stride = 0;
    if (!t) return nullptr;
    here(*t, name);
    TORCH_CHECK_VALUE(t->scalar_type() == type, name, " must be ", type, ", got ", t->scalar_type());
    TORCH_CHECK_VALUE(t->dim() == 2 && t->size(0) == n && t->size(1) == width, name,
                      " must have shape [", n, ", ", width, "], got ", t->sizes());
    TORCH_CHECK_VALUE(width <= 1 || t->stride(1) == 1, name,
                      ": the elements of a row must be contiguous");
    stride = n > 1 ? t->stride(0) : width;
    return t->data_ptr();
  }
};

int32_t dtype_of(at::ScalarType t, const char* name) {
  TORCH_CHECK_VALUE(t == at::kBFloat16 || t == at::kFloat, name,
                    " must be float32 or bfloat16, got ", t);
  return t == at::kFloat ? FDLLM_F32 : FDLLM_BF16;
}

// A size or index that fits the C argument.
int32_t as_int(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range: ", v);
  return (int32_t)v;
}

int32_t as_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return as_int(v, name);
}

PyObject* result(fdllm_status s) { return PyLong_FromLong(s); }

void expect(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

PyObject* item(PyObject* dict, const char* name) {
  PyObject* o = PyDict_GetItemString(dict, name);
  TORCH_CHECK_VALUE(o, "out has no ", name);
  return o;
}

// seq_lens, new_lens, block_table, page_size, free_pages, n_free, out, status
PyObject* plan_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor& table = needed(a[2], "block_table");
  const Call call(table, "block_table");
  TORCH_CHECK_VALUE(table.dim() == 2, "block_table must have two dimensions");
  TORCH_CHECK_TYPE(PyDict_Check(a[6]), "out must be a dict");
  const int64_t B = table.size(0), mb = table.size(1);
  const at::Tensor& free_pages = needed(a[4], "free_pages");
  const int64_t np = free_pages.numel();
  PyObject* pos = item(a[6], "positions");
  const int64_t cap = needed(pos, "positions").numel();
  auto wanted = [&](const char* name, int64_t size) {             // may be left out
    PyObject* o = PyDict_GetItemString(a[6], name);
    return call.i32<int32_t>(o ? o : Py_None, name, {size});
  };
  return result(plan_step_fn(
      as_int(B, "batch"), as_int(mb, "block_table's width"), as_int(a[3], "page_size"),
      as_int(np, "free_pages"), as_int(cap, "capacity"), call.i32<int32_t>(a[0], "seq_lens", {B}),
      call.i32<int32_t>(a[1], "new_lens", {B}), call.i32<int32_t>(a[2], "block_table", {B, mb}),
      call.i32<int32_t>(a[4], "free_pages", {np}), call.i32<int32_t>(a[5], "n_free", {1}),
      call.i32<int32_t>(item(a[6], "cu_rows"), "cu_rows", {B + 1}),
      call.i32<int32_t>(pos, "positions", {cap}),
      call.i32<int32_t>(item(a[6], "slots"), "slots", {cap}),
      call.i32<int32_t>(item(a[6], "row_seq"), "row_seq", {cap}),
      static_cast<int64_t*>(
          call.arg(tensor(item(a[6], "slot_map"), "slot_map"), "slot_map", at::kLong, {cap})),
      call.i32<int32_t>(item(a[6], "seq_lens"), "seq_lens (out)", {B}),
      call.i32<int32_t>(item(a[6], "granted"), "granted", {B}),
      call.i32<int32_t>(item(a[6], "n_free"), "n_free (out)", {1}),
      wanted("headroom", 1), wanted("seq_positions", B), wanted("seq_slots", B),
      call.i32<int32_t>(a[7], "status", {1}), call.stream()));
  END_HANDLE_TH_ERRORS
}

// seq_lens, keep_lens, block_table, page_size, free_pages, n_free, out, status
PyObject* release_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor& table = needed(a[2], "block_table");
  const Call call(table, "block_table");
  TORCH_CHECK_VALUE(table.dim() == 2, "block_table must have two dimensions");
  TORCH_CHECK_TYPE(PyDict_Check(a[6]), "out must be a dict");
  const int64_t B = table.size(0), mb = table.size(1);
  const int64_t np = needed(a[4], "free_pages").numel();
  return result(release_blocks_fn(
      as_int(B, "batch"), as_int(mb, "block_table's width"), as_int(a[3], "page_size"),
      as_int(np, "free_pages"), call.i32<int32_t>(a[0], "seq_lens", {B}),
      call.i32<int32_t>(a[1], "keep_lens", {B}), call.i32<int32_t>(a[2], "block_table", {B, mb}),
      call.i32<int32_t>(a[4], "free_pages", {np}), call.i32<int32_t>(a[5], "n_free", {1}),
      call.i32<int32_t>(item(a[6], "seq_lens"), "seq_lens (out)", {B}),
      call.i32<int32_t>(item(a[6], "n_free"), "n_free (out)", {1}),
      call.i32<int32_t>(a[7], "status", {1}), call.stream()));
  END_HANDLE_TH_ERRORS
}

// q, k_pool, v_pool, layer, block_table, seq_lens, k, v, positions, slots,
// rope_cos, rope_sin, starts, scale, out, out_f32, lse, with_lse, workspace,
// status -> (status, out, lse)
PyObject* decode_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 20);
  const at::Tensor& k_pool = needed(a[1], "k_pool");
  const Call call(k_pool, "k_pool");
  TORCH_CHECK_VALUE(k_pool.dim() == 5, "k_pool must have five dimensions");
  const at::Tensor &q = needed(a[0], "q"), &v_pool = needed(a[2], "v_pool"),
                   &table = needed(a[4], "block_table");
  const at::Tensor *k = tensor(a[6], "k"), *v = tensor(a[7], "v");
  const int64_t hk = k_pool.size(2), D = k_pool.size(4);
  TORCH_CHECK_VALUE(q.dim() == 2 && D > 0 && q.size(1) % D == 0,
                    "q must be [batch, n_heads * ", D, "], got ", q.sizes());
  const int64_t B = q.size(0), width = q.size(1), heads = width / D;
  TORCH_CHECK_VALUE(table.dim() == 2, "block_table must have two dimensions");
  const int64_t mb = table.size(1);

  at::Tensor out, lse, workspace;
  if (const at::Tensor* t = tensor(a[14], "out")) out = *t;
  else out = call.empty({B, width}, a[15] == Py_True ? at::kFloat : at::kBFloat16);
  if (const at::Tensor* t = tensor(a[16], "lse")) lse = *t;
  else if (a[17] == Py_True) lse = call.empty({B, heads}, at::kFloat);
  fdllm_status status = FDLLM_OK;
  if (B > 0) {
    fdllm_decode d = {};
    d.batch = as_int(B, "batch");
    d.n_heads = as_int(heads, "n_heads");
    d.n_kv_heads = as_int(hk, "n_kv_heads");
    d.head_dim = as_int(D, "head_dim");
    d.n_layers = as_int(k_pool.size(0), "n_layers");
    d.num_pages = as_int(k_pool.size(1), "num_pages");
    d.page_size = as_int(k_pool.size(3), "page_size");
    d.max_blocks_per_seq = as_int(mb, "block_table's width");
    d.dtype = dtype_of(k_pool.scalar_type(), "k_pool");
    d.in_dtype = dtype_of(q.scalar_type(), "q");
    d.out_dtype = dtype_of(out.scalar_type(), "out");
    d.scale = a[13] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)PyFloat_AsDouble(a[13]);
    if (PyErr_Occurred()) throw python_error();
    const at::Tensor *cos = tensor(a[10], "rope_cos"), *sin = tensor(a[11], "rope_sin");
    const int64_t positions = cos && cos->dim() == 2 ? cos->size(0) : 0;
    d.max_position = as_int(positions, "max_position");
    const void* qp = call.rows(&q, "q", q.scalar_type(), B, width, d.q_stride);
    const void* kp = call.rows(k, "k", q.scalar_type(), B, hk * D, d.k_stride);
    const void* vp = call.rows(v, "v", q.scalar_type(), B, hk * D, d.v_stride);
    int64_t bytes = 0;
    if (const at::Tensor* t = tensor(a[18], "workspace")) {
      workspace = *t;
      bytes = workspace.numel();
    } else {
      bytes = workspace_fn(d.n_heads, d.n_kv_heads, d.head_dim);
      workspace = call.empty({bytes > 16 ? bytes : 16}, at::kByte);
    }
    status = decode_fn(
        &d, as_int(a[3], "layer"), qp, kp, vp, call.i32<int32_t>(a[8], "positions", {B}),
        call.i32<int32_t>(a[9], "slots", {B}),
        static_cast<const double*>(call.arg(cos, "rope_cos", at::kDouble, {positions, D / 2})),
        static_cast<const double*>(call.arg(sin, "rope_sin", at::kDouble, {positions, D / 2})),
        call.arg(&k_pool, "k_pool", k_pool.scalar_type(), k_pool.sizes()),
        call.arg(&v_pool, "v_pool", k_pool.scalar_type(), k_pool.sizes()),
        call.i32<int32_t>(a[4], "block_table", {B, mb}), call.i32<int32_t>(a[5], "seq_lens", {B}),
        call.i32<int32_t>(a[12], "starts", {B}),
        call.arg(&out, "out", out.scalar_type(), {B, width}),
        static_cast<float*>(
            call.arg(lse.defined() ? &lse : nullptr, "lse", at::kFloat, {B, heads})),
        call.arg(&workspace, "workspace", at::kByte, {workspace.numel()}), bytes,
        call.i32<int32_t>(a[19], "status", {1}), call.stream());
  }
  PyObject* o = a[14] != Py_None ? (Py_INCREF(a[14]), a[14]) : THPVariable_Wrap(std::move(out));
  PyObject* l = a[16] != Py_None ? (Py_INCREF(a[16]), a[16])
                : lse.defined()  ? THPVariable_Wrap(std::move(lse))
                                 : (Py_INCREF(Py_None), Py_None);
  PyObject* r = PyTuple_New(3);
  PyTuple_SET_ITEM(r, 0, result(status));
  PyTuple_SET_ITEM(r, 1, o);
  PyTuple_SET_ITEM(r, 2, l);
  return r;
  END_HANDLE_TH_ERRORS
}

// x, w, bias, act, w_gate, bias_gate, residual, y, out_f32, status
// -> (status, y)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 10);
  const at::Tensor& x = needed(a[0], "x");
  const Call call(x, "x");
  const at::Tensor& w = needed(a[1], "w");
  TORCH_CHECK_VALUE(x.dim() == 2 && w.dim() == 2, "x and w must have two dimensions");
  const int64_t rows = x.size(0), n_in = x.size(1), n_out = w.size(1);
  const at::Tensor *bias = tensor(a[2], "bias"), *bias_gate = tensor(a[5], "bias_gate");
  const at::Tensor *w_gate = tensor(a[4], "w_gate"), *residual = tensor(a[6], "residual");
  at::Tensor y;
  if (const at::Tensor* t = tensor(a[7], "y")) y = *t;
  else y = call.empty({rows, n_out}, a[8] == Py_True ? at::kFloat : at::kBFloat16);
  const at::Tensor* b = bias ? bias : bias_gate;
  const at::ScalarType kind = b ? b->scalar_type() : at::kBFloat16;
  fdllm_linear_shape s = {};
  s.rows = as_int(rows, "rows");
  s.n_in = as_int(n_in, "n_in");
  s.n_out = as_int(n_out, "n_out");
  s.act = as_int(a[3], "act");
  s.bias_dtype = dtype_of(kind, "bias");
  s.out_dtype = dtype_of(y.scalar_type(), "y");
  const void* xp = call.rows(&x, "x", at::kBFloat16, rows, n_in, s.ldx);
  const void* rp = call.rows(residual, "residual", at::kBFloat16, rows, n_out, s.ldr);
  void* yp = call.rows(&y, "y", y.scalar_type(), rows, n_out, s.ldy);
  const fdllm_status status = linear_fn(
      &s, xp, call.arg(&w, "w", at::kBFloat16, {n_in, n_out}), call.arg(bias, "bias", kind, {n_out}),
      call.arg(w_gate, "w_gate", at::kBFloat16, {n_in, n_out}),
      call.arg(bias_gate, "bias_gate", kind, {n_out}), rp, yp,
      call.i32<int32_t>(a[9], "status", {1}), call.stream());
  PyObject* o = a[7] != Py_None ? (Py_INCREF(a[7]), a[7]) : THPVariable_Wrap(std::move(y));
  PyObject* r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, result(status));
  PyTuple_SET_ITEM(r, 1, o);
  return r;
  END_HANDLE_TH_ERRORS
}

// The library's entry points, by address.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 5);
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) throw python_error();
  }
  plan_step_fn = reinterpret_cast<decltype(plan_step_fn)>(p[0]);
  release_blocks_fn = reinterpret_cast<decltype(release_blocks_fn)>(p[1]);
  workspace_fn = reinterpret_cast<decltype(workspace_fn)>(p[2]);
  decode_fn = reinterpret_cast<decltype(decode_fn)>(p[3]);
  linear_fn = reinterpret_cast<decltype(linear_fn)>(p[4]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"), method<plan_blocks>("plan_blocks"),
                         method<release_blocks>("release_blocks"),
                         method<decode_attention>("decode_attention"), method<linear>("linear"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve() { return PyModule_Create(&module_def); }
