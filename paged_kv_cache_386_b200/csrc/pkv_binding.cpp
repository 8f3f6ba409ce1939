// pkv_binding.cpp -- the quick way from torch tensors to the C entry points whose
// calls are host-bound at a decode step's sizes (CPython extension `_binding`).
//
// Each function takes the plain case -- ordinary CUDA tensors on the current
// device and stream, with the types, shapes and strides that the entry point
// wants -- and returns NotImplemented for any other, also where the entry point
// refuses: the Python function of the same name then checks, reports and
// handles the call.  Measured for one token's rotating append, 24 arguments:
// 3.8 us of host time (launch 2.2, output 1.0, checks 0.6), and 13.4 through
// ctypes, of which 7.5 are checks in Python.
#include <Python.h>

#include <cstdint>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pagedkv.h"

namespace {

decltype(&paged_kv_append_rope) g_append_rope = nullptr;
decltype(&paged_kv_append_rope_fp8) g_append_rope_fp8 = nullptr;
decltype(&paged_kv_append_fp8) g_append_fp8 = nullptr;
decltype(&paged_attention_decode_fp8) g_decode_fp8 = nullptr;

constexpr int64_t kBlockTokens = 16;

PyObject* not_this() {
  Py_INCREF(Py_NotImplemented);
  return Py_NotImplemented;
}

// Other Python threads run while memory is allocated and the kernel launched: a
// full launch queue waits for the GPU, which may wait for a host function in Python.
struct WithoutGil {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

// The current device, or -1 where `obj` is no plain CUDA tensor (nothing of CUDA is touched then).
int device_for(PyObject* obj) {
  if (!THPVariable_CheckExact(obj) || !THPVariable_Unpack(obj).is_cuda()) return -1;
  return c10::cuda::current_device();
}

// A plain CUDA tensor on `device` (None: an undefined tensor, where that is allowed).
bool take(PyObject* obj, int device, at::Tensor* out, bool optional = false) {
  if (optional && obj == Py_None) return true;
  if (!THPVariable_CheckExact(obj)) return false;
  *out = THPVariable_Unpack(obj);
  return out->is_cuda() && out->get_device() == device;
}

bool dtype_of(const at::Tensor& t, pkv_dtype* dt) {
  switch (t.scalar_type()) {
    case at::kFloat: *dt = PKV_F32; return true;
    case at::kHalf: *dt = PKV_F16; return true;
    case at::kBFloat16: *dt = PKV_BF16; return true;
    default: return false;
  }
}

bool flat(const at::Tensor& t, at::ScalarType type, at::IntArrayRef sizes) {
  return t.scalar_type() == type && t.sizes() == sizes && t.is_contiguous();
}

// [n][h][d] with the heads of a token contiguous; the token stride in elements.
bool heads(const at::Tensor& t, at::ScalarType type, int64_t n, int64_t h, int64_t d, int64_t* stride) {
  if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != n || t.size(1) != h || t.size(2) != d ||
      t.stride(2) != 1 || t.stride(1) != d)
    return false;
  *stride = n > 1 ? t.stride(0) : h * d;
  return true;
}

// The cache's blocks and kv heads; `second` is the V cache, or the FP8 cache's scales.
bool cache_of(const at::Tensor& cache, const at::Tensor& second, bool fp8, at::ScalarType type, int64_t d, int64_t* nb,
              int64_t* n_kv) {
  if (cache.dim() != (fp8 ? 5 : 4)) return false;
  *nb = cache.size(0);
  *n_kv = cache.size(1);
  if (fp8)
    return flat(cache, at::kFloat8_e4m3fn, {*nb, *n_kv, 2, kBlockTokens, d}) && flat(second, at::kFloat, {*nb, *n_kv, 2});
  return flat(cache, type, {*nb, *n_kv, kBlockTokens, d}) && flat(second, type, {*nb, *n_kv, kBlockTokens, d});
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// append_rope(k, v, positions, cos_sin, slot_mapping, cache, second, q, q_out, interleaved, fp8) -> q_out or None
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  const int device = n_args == 11 ? device_for(a[0]) : -1;
  if (device < 0) return not_this();
  at::Tensor k, v, pos, table, slots, cache, second, q, q_out;
  if (!take(a[0], device, &k) || !take(a[1], device, &v) || !take(a[2], device, &pos) || !take(a[3], device, &table) ||
      !take(a[4], device, &slots) || !take(a[5], device, &cache) || !take(a[6], device, &second) ||
      !take(a[7], device, &q, true) || !take(a[8], device, &q_out, true))
    return not_this();
  const int interleaved = PyObject_IsTrue(a[9]), fp8 = PyObject_IsTrue(a[10]);
  if (interleaved < 0 || fp8 < 0) return nullptr;
  pkv_dtype dt;
  if (k.dim() != 3 || !dtype_of(k, &dt) || table.dim() != 2) return not_this();
  const at::ScalarType type = k.scalar_type();
  const int64_t n = k.size(0), d = k.size(2);
  int64_t nb, n_kv, ks, vs, qs = 0, os = 0, n_q = 0;
  if (!cache_of(cache, second, fp8 != 0, type, d, &nb, &n_kv) || !heads(k, type, n, n_kv, d, &ks) ||
      !heads(v, type, n, n_kv, d, &vs) || !flat(slots, at::kLong, {n}) || !flat(pos, at::kLong, {n}) ||
      !flat(table, at::kFloat, table.sizes()) || n > INT32_MAX || nb > INT32_MAX || table.size(1) > INT32_MAX ||
      n_kv > INT32_MAX || d > INT32_MAX)
    return not_this();
  if (q.defined()) {
    if (q.dim() != 3) return not_this();
    n_q = q.size(1);
    if (n_q > INT32_MAX) return not_this();
    if (!heads(q, type, n, n_q, d, &qs)) return not_this();
    os = n_q * d;
    if (q_out.defined() && !heads(q_out, type, n, n_q, d, &os)) return not_this();
  } else if (q_out.defined()) {
    return not_this();
  }
  const void* qp = q.defined() ? q.data_ptr() : nullptr;
  const int32_t rot = static_cast<int32_t>(table.size(1)), n32 = static_cast<int32_t>(n), nb32 = static_cast<int32_t>(nb),
                nq32 = static_cast<int32_t>(n_q), nkv32 = static_cast<int32_t>(n_kv), d32 = static_cast<int32_t>(d);
  const int64_t* pp = pos.data_ptr<int64_t>();
  const int64_t* sp = slots.data_ptr<int64_t>();
  const float* tp = table.data_ptr<float>();
  pkv_status st;
  {
    WithoutGil released;
    if (q.defined() && !q_out.defined()) q_out = at::detail::empty_cuda({n, n_q, d}, type, q.device(), std::nullopt);
    void* op = q_out.defined() ? q_out.data_ptr() : nullptr;
    if (fp8)
      st = g_append_rope_fp8(qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, pp, tp, table.size(0), rot, interleaved, sp, n32,
                             static_cast<uint8_t*>(cache.data_ptr()), second.data_ptr<float>(), nb32, kBlockTokens, nq32,
                             nkv32, d32, op, os, dt, stream_of(device));
    else
      st = g_append_rope(qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, pp, tp, table.size(0), rot, interleaved, sp, n32,
                         cache.data_ptr(), second.data_ptr(), nb32, kBlockTokens, nq32, nkv32, d32, op, os, dt,
                         stream_of(device));
  }
  if (st != PKV_OK) return not_this();
  if (!q.defined()) Py_RETURN_NONE;
  if (a[8] != Py_None) {
    Py_INCREF(a[8]);
    return a[8];
  }
  return THPVariable_Wrap(std::move(q_out));
  END_HANDLE_TH_ERRORS
}

// append_fp8(k, v, slot_mapping, kv_cache, kv_scales) -> None
PyObject* append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  const int device = n_args == 5 ? device_for(a[0]) : -1;
  if (device < 0) return not_this();
  at::Tensor k, v, slots, cache, scales;
  if (!take(a[0], device, &k) || !take(a[1], device, &v) || !take(a[2], device, &slots) || !take(a[3], device, &cache) ||
      !take(a[4], device, &scales))
    return not_this();
  pkv_dtype dt;
  if (k.dim() != 3 || !dtype_of(k, &dt)) return not_this();
  const int64_t n = k.size(0), d = k.size(2);
  int64_t nb, n_kv, ks, vs;
  if (!cache_of(cache, scales, true, k.scalar_type(), d, &nb, &n_kv) || !heads(k, k.scalar_type(), n, n_kv, d, &ks) ||
      !heads(v, k.scalar_type(), n, n_kv, d, &vs) || !flat(slots, at::kLong, {n}) || n > INT32_MAX || nb > INT32_MAX ||
      n_kv > INT32_MAX || d > INT32_MAX)
    return not_this();
  pkv_status st;
  {
    WithoutGil released;
    st = g_append_fp8(k.data_ptr(), ks, v.data_ptr(), vs, dt, slots.data_ptr<int64_t>(), static_cast<int32_t>(n),
                      static_cast<uint8_t*>(cache.data_ptr()), scales.data_ptr<float>(), static_cast<int32_t>(nb),
                      kBlockTokens, static_cast<int32_t>(n_kv), static_cast<int32_t>(d), stream_of(device));
  }
  if (st != PKV_OK) return not_this();
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// decode_fp8(q, kv_cache, kv_scales, block_tables, context_lens, scale, out, workspace) -> out
PyObject* decode_fp8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  const int device = n_args == 8 && PyFloat_CheckExact(a[5]) ? device_for(a[0]) : -1;
  if (device < 0) return not_this();
  at::Tensor q, cache, scales, tables, lens, out, ws;
  if (!take(a[0], device, &q) || !take(a[1], device, &cache) || !take(a[2], device, &scales) ||
      !take(a[3], device, &tables) || !take(a[4], device, &lens) || !take(a[6], device, &out, true) ||
      !take(a[7], device, &ws, true))
    return not_this();
  pkv_dtype dt;
  if ((q.dim() != 3 && q.dim() != 4) || !dtype_of(q, &dt) || !q.is_contiguous() || tables.dim() != 2) return not_this();
  const int64_t batch = q.size(0), q_len = q.dim() == 4 ? q.size(1) : 1, n_q = q.size(-2), d = q.size(-1);
  int64_t nb, n_kv;
  if (!cache_of(cache, scales, true, at::kFloat, d, &nb, &n_kv) || !flat(tables, at::kInt, {batch, tables.size(1)}) ||
      !flat(lens, at::kInt, {batch}) || (out.defined() && !flat(out, q.scalar_type(), q.sizes())) ||
      (ws.defined() && !ws.is_contiguous()) || batch > INT32_MAX || q_len > INT32_MAX || n_q > INT32_MAX ||
      nb > INT32_MAX || tables.size(1) > INT32_MAX ||
      n_kv > INT32_MAX || d > INT32_MAX)
    return not_this();
  const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[5]));
  pkv_status st;
  {
    WithoutGil released;
    if (!out.defined()) out = at::detail::empty_cuda(q.sizes(), q.scalar_type(), q.device(), std::nullopt);
    st = g_decode_fp8(q.data_ptr(), static_cast<const uint8_t*>(cache.data_ptr()), scales.data_ptr<float>(),
                      tables.data_ptr<int32_t>(), static_cast<int32_t>(tables.size(1)), lens.data_ptr<int32_t>(),
                      static_cast<int32_t>(batch), static_cast<int32_t>(q_len), static_cast<int32_t>(nb), scale,
                      static_cast<int32_t>(n_q), static_cast<int32_t>(n_kv), static_cast<int32_t>(d), kBlockTokens,
                      out.data_ptr(), dt, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                      stream_of(device));
  }
  if (st != PKV_OK) return not_this();
  if (a[6] != Py_None) {
    Py_INCREF(a[6]);
    return a[6];
  }
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of paged_kv_append_rope, paged_kv_append_rope_fp8, paged_kv_append_fp8, paged_attention_decode_fp8)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "KKKK", &f[0], &f[1], &f[2], &f[3])) return nullptr;
  g_append_rope = reinterpret_cast<decltype(g_append_rope)>(f[0]);
  g_append_rope_fp8 = reinterpret_cast<decltype(g_append_rope_fp8)>(f[1]);
  g_append_fp8 = reinterpret_cast<decltype(g_append_fp8)>(f[2]);
  g_decode_fp8 = reinterpret_cast<decltype(g_decode_fp8)>(f[3]);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_rope)), METH_FASTCALL, nullptr},
    {"append_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_fp8)), METH_FASTCALL, nullptr},
    {"decode_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_fp8)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", PKV_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
