// torch_calls.cpp -- the torch side of the feed-forward calls, the grouped
// products and the adapters, as a CPython module: argument checks, allocation of
// results, and one call into the C ABI.
//
// A decoding step makes these calls for 2-15 us of GPU work each, so what the
// host spends on them counts.  Host time of a call at 16 x 64 x 64, written in
// Python over ctypes and here: gated 8.8 and 4.3 us, with both projections
// stored 11.9 and 5.7, the 8-bit product 9.2 and 4.2, quantization 8.3 and 4.4,
// the backward pass (four launches) 21.6 and 11.4; here alone: a grouped product
// 4.5, one row with an adapter 5.3, eight (two launches) 7.3, a grouped product and
// its two gradients 12.  Two thirds and more of what
// is left are the launches themselves.  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "tg_gemm.h"

namespace {

PyObject* g_error = nullptr;  // the package's TGError

// Raise TGError(status, what) for a status that is not TG_OK.
void check_status(int status, const char* what) {
  if (status == TG_OK) return;
  PyObject* value = PyObject_CallFunction(g_error, "is", status, what);
  if (value) {
    PyErr_SetObject(g_error, value);
    Py_DECREF(value);
  }
  throw python_error();
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  // A view whose values are the negatives of its memory (the imaginary part of a conjugate).
  TORCH_CHECK_VALUE(!t.is_neg(), name, " is a negated view; pass its resolve_neg()");
  return t;
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  const at::Tensor& t = tensor_of(o, name);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
  return t;
}

int type_code(at::ScalarType t) {
  TORCH_CHECK_TYPE(t == at::kHalf || t == at::kBFloat16, "expected torch.float16 or torch.bfloat16, got ", t);
  return t == at::kHalf ? TG_TYPE_F16 : TG_TYPE_BF16;
}

int act_code(PyObject* act) {
  if (PyUnicode_Check(act)) {
    if (PyUnicode_CompareWithASCIIString(act, "silu") == 0) return TG_ACT_SILU;
    if (PyUnicode_CompareWithASCIIString(act, "gelu") == 0) return TG_ACT_GELU;
    if (PyUnicode_CompareWithASCIIString(act, "relu") == 0) return TG_ACT_RELU;
  }
  TORCH_CHECK_VALUE(false, "unknown activation; one of 'gelu', 'relu', 'silu'");
}

// A tensor (..., cols) as rows: ld elements apart, 0 for dense rows or a single one.
struct Rows {
  int64_t rows, cols, ld;
};

Rows rows_of(const at::Tensor& t, const char* name) {
  const int64_t d = t.dim();
  TORCH_CHECK_VALUE(d >= 1, name, " needs at least one dimension");
  Rows r{1, t.size(d - 1), 0};
  for (int64_t i = 0; i < d - 1; ++i) r.rows *= t.size(i);
  if (t.is_contiguous() || r.rows == 0 || r.cols == 0) return r;
  TORCH_CHECK_VALUE(r.cols == 1 || t.stride(d - 1) == 1, name, " must have adjacent columns (stride 1), got strides ",
                    t.strides());
  int64_t span = 0;
  for (int64_t i = d - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (span == 0) {
      r.ld = t.stride(i);
      TORCH_CHECK_VALUE(r.ld >= r.cols, name, " has overlapping rows: strides ", t.strides(), " for shape ", t.sizes());
    } else {
      TORCH_CHECK_VALUE(t.stride(i) == span, name, ": the leading dimensions of shape ", t.sizes(), " with strides ",
                        t.strides(), " are not evenly spaced rows");
    }
    span = t.stride(i) * t.size(i);
  }
  return r;
}

// The row stride of an operand that has to have this shape, type and device.
int64_t matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, at::ScalarType type,
               const at::Device& device, bool two_dimensional = true) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", got ", t.device());
  if (two_dimensional)
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols, name, " must have shape (", rows, ", ",
                      cols, "), got ", t.sizes());
  const Rows r = rows_of(t, name);
  TORCH_CHECK_VALUE(r.rows == rows && r.cols == cols, name, " must have ", rows, " rows of ", cols, ", got shape ",
                    t.sizes());
  return r.ld;
}

const void* vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type, const at::Device& device) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.numel() == n && t.is_contiguous() && t.device() == device, name, " must be ", n,
                    " contiguous values on ", device);
  return t.data_ptr();
}

// A new tensor with x's leading dimensions and `cols` columns, rows `ld` elements apart (0: dense).
at::Tensor new_rows(const at::Tensor& x, int64_t cols, int64_t ld, at::ScalarType type) {
  const int64_t d = x.dim();
  if (ld == 0 || ld == cols) {
    if (d == 2) return at::detail::empty_cuda({x.size(0), cols}, type, x.device(), std::nullopt);
    std::vector<int64_t> sizes(x.sizes().begin(), x.sizes().end());
    sizes[d - 1] = cols;
    return at::detail::empty_cuda(sizes, type, x.device(), std::nullopt);
  }
  std::vector<int64_t> sizes(x.sizes().begin(), x.sizes().end()), strides(d);
  sizes[d - 1] = cols;
  strides[d - 1] = 1;
  int64_t step = ld;
  for (int64_t i = d - 2; i >= 0; --i) {
    strides[i] = step;
    step *= sizes[i];
  }
  return at::detail::empty_strided_cuda(sizes, strides, type, x.device());
}

// The given result, checked to have x's leading dimensions and `cols` columns; its row stride.
const at::Tensor& given_rows(PyObject* o, const char* name, const at::Tensor& x, int64_t rows, int64_t cols,
                             at::ScalarType type, int64_t* ld) {
  const at::Tensor& t = tensor_of(o, name);
  const int64_t d = x.dim();
  TORCH_CHECK_VALUE(t.dim() == d && t.sizes().slice(0, d - 1) == x.sizes().slice(0, d - 1) && t.size(d - 1) == cols,
                    name, " must have the leading dimensions of ", x.sizes(), " and ", cols, " columns, got ", t.sizes());
  *ld = matrix(t, name, rows, cols, type, x.device(), false);
  return t;
}

// The workspace of a call that needs `need` bytes: torch's ("auto"), none, or the given tensor.
struct Scratch {
  at::Tensor held;
  void* ptr = nullptr;
  int64_t bytes = 0;

  Scratch(PyObject* o, int64_t need, const at::Device& device) {
    check_status(need < 0 ? TG_ERR_INVALID_ARG : TG_OK, "workspace size");
    if (o == Py_None) return;
    if (PyUnicode_Check(o)) {
      TORCH_CHECK_VALUE(PyUnicode_CompareWithASCIIString(o, "auto") == 0,
                        "workspace must be 'auto', None or a uint8 CUDA tensor");
      if (need == 0) return;
      held = at::detail::empty_cuda({need}, at::kByte, device, std::nullopt);
    } else {
      held = tensor_of(o, "workspace");
      TORCH_CHECK_VALUE(held.scalar_type() == at::kByte && held.is_contiguous() && held.device() == device,
                        "workspace must be a contiguous uint8 tensor on ", device);
    }
    ptr = held.data_ptr();
    bytes = held.numel();
  }
};

void* stream_of(const at::Device& device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

// Launches may wait for room in a stream's queue: other host threads run meanwhile.
struct WithoutGil {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

template <typename Call>
void call(const char* what, Call&& c) {
  int status;
  {
    WithoutGil no_gil;
    status = c();
  }
  check_status(status, what);
}

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw python_error();
  return t == 1;
}

PyObject* new_ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// The caller's tensor as a result: its version counts up, so that a backward pass that saved its old values says so.
PyObject* written(PyObject* o) {
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return new_ref(o);
}

// (a, b, c), taking over the references.
template <typename... Items>
PyObject* tuple_of(Items... items) {
  PyObject* t = PyTuple_New(sizeof...(items));
  if (!t) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(t, i++, items), ...);
  return t;
}

void want_args(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// gated(x, w_gate, w_up, act, out, save, workspace)
PyObject* gated(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 7);
  const at::Tensor& x = cuda_tensor(args[0], "x");
  const at::Tensor &wg = tensor_of(args[1], "w_gate"), &wu = tensor_of(args[2], "w_up");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType type = x.scalar_type();
  const Rows xr = rows_of(x, "x");
  tg_gated_options o{};
  o.type = type_code(type);
  o.act = act_code(args[3]);
  TORCH_CHECK_VALUE(wg.dim() == 2, "w_gate must be (N, K), got ", wg.sizes());
  const int64_t M = xr.rows, K = xr.cols, N = wg.size(0);
  o.ldx = xr.ld;
  o.ldwg = matrix(wg, "w_gate", N, K, type, device);
  o.ldwu = matrix(wu, "w_up", N, K, type, device);
  const bool given = args[4] != Py_None, save = truth(args[5]);
  const at::Tensor out =
      given ? given_rows(args[4], "out", x, M, N, type, &o.ldh) : new_rows(x, N, 0, type);
  at::Tensor gate, up;
  if (save) {
    // Rows of the stored projections start on 16-byte boundaries whatever N is: they leave by TMA and come
    // back in whole vectors (forward of 2000 x 4095 x 2047 with both stored: 84 us dense, 73 us so).
    o.ldg = o.ldu = (N + 7) / 8 * 8;
    gate = new_rows(x, N, o.ldg, type);
    up = new_rows(x, N, o.ldu, type);
  }
  const void *px = x.data_ptr(), *pg = wg.data_ptr(), *pu = wu.data_ptr();
  const Scratch ws(args[6], tg_gated_workspace_size(px, pg, pu, M, N, K, &o), device);
  call("tg_gated", [&] {
    return tg_gated(px, pg, pu, out.data_ptr(), save ? gate.data_ptr() : nullptr, save ? up.data_ptr() : nullptr, M, N,
                    K, &o, stream_of(device), ws.ptr, ws.bytes);
  });
  PyObject* result = given ? written(args[4]) : THPVariable_Wrap(out);
  return save ? tuple_of(result, THPVariable_Wrap(gate), THPVariable_Wrap(up)) : result;
  END_HANDLE_TH_ERRORS
}

// gated_backward(grad, x, w_gate, w_up, gate, up, act, need_x, need_gate, need_up, workspace)
PyObject* gated_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 11);
  const at::Tensor& x = cuda_tensor(args[1], "x");
  const at::Tensor &grad = tensor_of(args[0], "grad"), &wg = tensor_of(args[2], "w_gate"),
                   &wu = tensor_of(args[3], "w_up"), &gate = tensor_of(args[4], "gate"), &up = tensor_of(args[5], "up");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType type = x.scalar_type();
  const Rows xr = rows_of(x, "x");
  tg_gated_options o{};
  o.type = type_code(type);
  o.act = act_code(args[6]);
  TORCH_CHECK_VALUE(wg.dim() == 2, "w_gate must be (N, K), got ", wg.sizes());
  const int64_t M = xr.rows, K = xr.cols, N = wg.size(0);
  o.ldx = xr.ld;
  o.ldwg = matrix(wg, "w_gate", N, K, type, device);
  o.ldwu = matrix(wu, "w_up", N, K, type, device);
  o.ldh = matrix(grad, "grad", M, N, type, device, false);
  o.ldg = matrix(gate, "gate", M, N, type, device, false);
  o.ldu = matrix(up, "up", M, N, type, device, false);
  at::Tensor dx, dwg, dwu;
  if (truth(args[7])) dx = new_rows(x, K, 0, type);
  if (truth(args[8])) dwg = at::detail::empty_cuda({N, K}, type, device, std::nullopt);
  if (truth(args[9])) dwu = at::detail::empty_cuda({N, K}, type, device, std::nullopt);
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  auto wrap = [](const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : new_ref(Py_None); };
  const void *px = x.data_ptr(), *pg = wg.data_ptr(), *pu = wu.data_ptr();
  const Scratch ws(args[10], tg_gated_backward_workspace_size(px, pg, pu, ptr(dx), ptr(dwg), ptr(dwu), M, N, K, &o),
                   device);
  call("tg_gated_backward", [&] {
    return tg_gated_backward(grad.data_ptr(), px, pg, pu, gate.data_ptr(), up.data_ptr(), ptr(dx), ptr(dwg), ptr(dwu),
                             M, N, K, &o, stream_of(device), ws.ptr, ws.bytes);
  });
  return tuple_of(wrap(dx), wrap(dwg), wrap(dwu));
  END_HANDLE_TH_ERRORS
}

// quantize_i8(x, out, scales)
PyObject* quantize_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 3);
  const at::Tensor& x = cuda_tensor(args[0], "x");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const int type = type_code(x.scalar_type());
  const Rows r = rows_of(x, "x");
  const bool given_q = args[1] != Py_None, given_s = args[2] != Py_None;
  int64_t ldq = (r.cols + 15) / 16 * 16;
  const at::Tensor q = given_q ? given_rows(args[1], "out", x, r.rows, r.cols, at::kChar, &ldq)
                               : new_rows(x, r.cols, ldq, at::kChar);
  at::Tensor s;
  if (given_s) {
    s = tensor_of(args[2], "scales");
    vector(s, "scales", r.rows, at::kFloat, device);
  } else {
    s = at::detail::empty_cuda(x.sizes().slice(0, x.dim() - 1), at::kFloat, device, std::nullopt);
  }
  call("tg_quantize_rows_i8", [&] {
    return tg_quantize_rows_i8(x.data_ptr(), q.data_ptr(), static_cast<float*>(s.data_ptr()), r.rows, r.cols, r.ld,
                               ldq, type, stream_of(device));
  });
  return tuple_of(given_q ? written(args[1]) : THPVariable_Wrap(q), given_s ? written(args[2]) : THPVariable_Wrap(s));
  END_HANDLE_TH_ERRORS
}

// The type of an 8-bit product's result: the asked one, or out's, or float16.
at::ScalarType result_type(PyObject* dtype, PyObject* out) {
  if (dtype != Py_None) {
    TORCH_CHECK_TYPE(THPDtype_Check(dtype), "dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  }
  return out != Py_None ? tensor_of(out, "out").scalar_type() : at::kHalf;
}

// gemm_i8(a, a_scale, w, w_scale, bias, relu, dtype, out)
PyObject* gemm_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 8);
  const at::Tensor& a = cuda_tensor(args[0], "a");
  const at::Tensor &sa = tensor_of(args[1], "a_scale"), &w = tensor_of(args[2], "w"), &sw = tensor_of(args[3], "w_scale");
  const at::Device device = a.device();
  const c10::cuda::CUDAGuard guard(device);
  TORCH_CHECK_VALUE(w.dim() == 2, "w must be (N, K), got ", w.sizes());
  const Rows ar = rows_of(a, "a");
  const int64_t M = ar.rows, K = ar.cols, N = w.size(0);
  matrix(a, "a", M, K, at::kChar, device, false);
  const int64_t ldw = matrix(w, "w", N, K, at::kChar, device);
  const void *psa = vector(sa, "a_scale", M, at::kFloat, device), *psw = vector(sw, "w_scale", N, at::kFloat, device);
  const at::ScalarType type = result_type(args[6], args[7]);
  const int code = type_code(type);
  const void* bias = args[4] == Py_None ? nullptr : vector(tensor_of(args[4], "bias"), "bias", N, type, device);
  const bool given = args[7] != Py_None;
  const int relu = truth(args[5]) ? 1 : 0;
  int64_t ldc = 0;
  const at::Tensor out = given ? given_rows(args[7], "out", a, M, N, type, &ldc) : new_rows(a, N, 0, type);
  call("tg_gemm_i8", [&] {
    return tg_gemm_i8(a.data_ptr(), static_cast<const float*>(psa), w.data_ptr(), static_cast<const float*>(psw), bias,
                      out.data_ptr(), M, N, K, ar.ld, ldw, ldc, relu, code, stream_of(device));
  });
  return given ? written(args[7]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// gated_i8(a, a_scale, w_gate, gate_scale, w_up, up_scale, act, dtype, out)
PyObject* gated_i8(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 9);
  const at::Tensor& a = cuda_tensor(args[0], "a");
  const at::Tensor &sa = tensor_of(args[1], "a_scale"), &wg = tensor_of(args[2], "w_gate"),
                   &sg = tensor_of(args[3], "gate_scale"), &wu = tensor_of(args[4], "w_up"),
                   &su = tensor_of(args[5], "up_scale");
  const at::Device device = a.device();
  const c10::cuda::CUDAGuard guard(device);
  TORCH_CHECK_VALUE(wg.dim() == 2, "w_gate must be (N, K), got ", wg.sizes());
  const Rows ar = rows_of(a, "a");
  const int64_t M = ar.rows, K = ar.cols, N = wg.size(0);
  const at::ScalarType type = result_type(args[7], args[8]);
  tg_gated_options o{};
  o.type = type_code(type);
  o.act = act_code(args[6]);
  o.ldx = matrix(a, "a", M, K, at::kChar, device, false);
  o.ldwg = matrix(wg, "w_gate", N, K, at::kChar, device);
  o.ldwu = matrix(wu, "w_up", N, K, at::kChar, device);
  const float* psa = static_cast<const float*>(vector(sa, "a_scale", M, at::kFloat, device));
  const float* psg = static_cast<const float*>(vector(sg, "gate_scale", N, at::kFloat, device));
  const float* psu = static_cast<const float*>(vector(su, "up_scale", N, at::kFloat, device));
  const bool given = args[8] != Py_None;
  const at::Tensor out = given ? given_rows(args[8], "out", a, M, N, type, &o.ldh) : new_rows(a, N, 0, type);
  call("tg_gated_i8", [&] {
    return tg_gated_i8(a.data_ptr(), psa, wg.data_ptr(), psg, wu.data_ptr(), psu, out.data_ptr(), M, N, K, &o,
                       stream_of(device));
  });
  return given ? written(args[8]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// Strides of stacked matrices (n, rows, cols) of this type: between rows and between matrices, 0 for dense ones.
struct Stack {
  int64_t ld = 0, stride = 0;
};

Stack stack(const at::Tensor& t, const char* name, int64_t n, int64_t rows, int64_t cols, at::ScalarType type,
            const at::Device& device) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", got ", t.device());
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == n && t.size(1) == rows && t.size(2) == cols, name, " must have shape (", n,
                    ", ", rows, ", ", cols, "), got ", t.sizes());
  Stack s;
  if (t.is_contiguous() || t.numel() == 0) return s;
  TORCH_CHECK_VALUE((cols == 1 || t.stride(2) == 1) && (rows == 1 || t.stride(1) >= cols) && (n == 1 || t.stride(0) >= cols),
                    name, " must have adjacent columns and rows that do not overlap, got strides ", t.strides());
  if (rows > 1) s.ld = t.stride(1);
  if (n > 1) s.stride = t.stride(0);
  return s;
}

// grouped(x, w, ends, out, workspace)
PyObject* grouped(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 5);
  const at::Tensor& x = cuda_tensor(args[0], "x");
  const at::Tensor &w = tensor_of(args[1], "w"), &ends = tensor_of(args[2], "ends");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType type = x.scalar_type();
  const Rows xr = rows_of(x, "x");
  tg_grouped_options o{};
  o.type = type_code(type);
  TORCH_CHECK_VALUE(w.dim() == 3, "w must be (groups, N, K), got ", w.sizes());
  const int64_t G = w.size(0), M = xr.rows, K = xr.cols, N = w.size(1);
  o.ldx = xr.ld;
  const Stack ws3 = stack(w, "w", G, N, K, type, device);
  o.ldw = ws3.ld;
  o.stride_w = ws3.stride;
  const void* pe = vector(ends, "ends", G, at::kInt, device);
  const bool given = args[3] != Py_None;
  // A new result has defined rows throughout; a given one keeps those that belong to no group.
  o.rest = given ? 0 : 1;
  const at::Tensor out = given ? given_rows(args[3], "out", x, M, N, type, &o.ldy) : new_rows(x, N, 0, type);
  TORCH_CHECK_VALUE(G <= INT32_MAX, "too many groups");
  const int32_t groups = static_cast<int32_t>(G);
  const void *px = x.data_ptr(), *pw = w.data_ptr();
  const Scratch ws(args[4], tg_grouped_workspace_size(px, pw, groups, M, N, K, &o), device);
  call("tg_grouped", [&] {
    return tg_grouped(px, pw, static_cast<const int32_t*>(pe), out.data_ptr(), groups, M, N, K, &o, stream_of(device), ws.ptr,
                      ws.bytes);
  });
  return given ? written(args[3]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// grouped_backward(grad, x, w, ends, need_x, need_w, workspace)
PyObject* grouped_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 7);
  const at::Tensor& x = cuda_tensor(args[1], "x");
  const at::Tensor &grad = tensor_of(args[0], "grad"), &w = tensor_of(args[2], "w"), &ends = tensor_of(args[3], "ends");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType type = x.scalar_type();
  const Rows xr = rows_of(x, "x");
  tg_grouped_options o{};
  o.type = type_code(type);
  o.rest = 1;
  TORCH_CHECK_VALUE(w.dim() == 3, "w must be (groups, N, K), got ", w.sizes());
  const int64_t G = w.size(0), M = xr.rows, K = xr.cols, N = w.size(1);
  o.ldx = xr.ld;
  const Stack ws3 = stack(w, "w", G, N, K, type, device);
  o.ldw = ws3.ld;
  o.stride_w = ws3.stride;
  o.ldy = matrix(grad, "grad", M, N, type, device, false);
  const void* pe = vector(ends, "ends", G, at::kInt, device);
  TORCH_CHECK_VALUE(G <= INT32_MAX, "too many groups");
  const int32_t groups = static_cast<int32_t>(G);
  at::Tensor dx, dw;
  if (truth(args[4])) dx = new_rows(x, K, 0, type);
  if (truth(args[5])) dw = at::detail::empty_cuda({G, N, K}, type, device, std::nullopt);
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  auto wrap = [](const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : new_ref(Py_None); };
  const void *pd = grad.data_ptr(), *px = x.data_ptr(), *pw = w.data_ptr();
  const Scratch ws(args[6], tg_grouped_backward_workspace_size(pd, px, pw, ptr(dx), ptr(dw), groups, M, N, K, &o), device);
  call("tg_grouped_backward", [&] {
    return tg_grouped_backward(pd, px, pw, static_cast<const int32_t*>(pe), ptr(dx), ptr(dw), groups, M, N, K, &o,
                               stream_of(device), ws.ptr, ws.bytes);
  });
  return tuple_of(wrap(dx), wrap(dw));
  END_HANDLE_TH_ERRORS
}

// lora(x, w, a, b, index, scale, bias, out, workspace)
PyObject* lora(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  want_args(nargs, 9);
  const at::Tensor& x = cuda_tensor(args[0], "x");
  const at::Tensor &w = tensor_of(args[1], "w"), &a = tensor_of(args[2], "a"), &b = tensor_of(args[3], "b"),
                   &index = tensor_of(args[4], "index");
  const at::Device device = x.device();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType type = x.scalar_type();
  const Rows xr = rows_of(x, "x");
  tg_lora_options o{};
  o.type = type_code(type);
  TORCH_CHECK_VALUE(w.dim() == 2, "w must be (N, K), got ", w.sizes());
  TORCH_CHECK_VALUE(a.dim() == 3, "a must be (adapters, rank, K), got ", a.sizes());
  const int64_t M = xr.rows, K = xr.cols, N = w.size(0), R = a.size(0), rank = a.size(1);
  o.ldx = xr.ld;
  o.ldw = matrix(w, "w", N, K, type, device);
  const Stack sa = stack(a, "a", R, rank, K, type, device), sb = stack(b, "b", R, N, rank, type, device);
  o.lda = sa.ld;
  o.stride_a = sa.stride;
  o.ldb = sb.ld;
  o.stride_b = sb.stride;
  TORCH_CHECK_VALUE(rank % 8 == 0, "the adapters' rank must be a multiple of 8, got ", rank);
  const auto off16 = [&](const at::Tensor& t, const Stack& s, int64_t cols) {
    return t.numel() != 0 && (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0 || (s.ld ? s.ld : cols) % 8 != 0 || s.stride % 8 != 0);
  };
  TORCH_CHECK_VALUE(!off16(a, sa, K) && !off16(b, sb, rank), "rows of a and b must start on 16-byte boundaries");
  const void* pi = vector(index, "index", M, at::kInt, device);
  const float* ps = args[5] == Py_None ? nullptr
                                       : static_cast<const float*>(vector(tensor_of(args[5], "scale"), "scale", R, at::kFloat, device));
  const void* bias = args[6] == Py_None ? nullptr : vector(tensor_of(args[6], "bias"), "bias", N, type, device);
  const bool given = args[7] != Py_None;
  const at::Tensor out = given ? given_rows(args[7], "out", x, M, N, type, &o.ldy) : new_rows(x, N, 0, type);
  const void *px = x.data_ptr(), *pw = w.data_ptr();
  const Scratch ws(args[8], tg_lora_workspace_size(px, pw, M, N, K, rank, R, &o), device);
  call("tg_lora", [&] {
    return tg_lora(px, pw, a.data_ptr(), b.data_ptr(), ps, static_cast<const int32_t*>(pi), bias, out.data_ptr(), M, N, K, rank, R,
                   &o, stream_of(device), ws.ptr, ws.bytes);
  });
  return given ? written(args[7]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// has_tangent(tensors...): whether any is a dual tensor of forward-mode differentiation.
PyObject* has_tangent(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  for (Py_ssize_t i = 0; i < nargs; ++i) {
    TORCH_CHECK_TYPE(THPVariable_Check(args[i]), "expected tensors");
    if (THPVariable_Unpack(args[i])._fw_grad(/*level=*/0).defined()) Py_RETURN_TRUE;
  }
  Py_RETURN_FALSE;
  END_HANDLE_TH_ERRORS
}

// set_error(class): what a status that is not TG_OK is raised as.
PyObject* set_error(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"gated", fast(gated), METH_FASTCALL, nullptr},
    {"gated_backward", fast(gated_backward), METH_FASTCALL, nullptr},
    {"quantize_i8", fast(quantize_i8), METH_FASTCALL, nullptr},
    {"gemm_i8", fast(gemm_i8), METH_FASTCALL, nullptr},
    {"gated_i8", fast(gated_i8), METH_FASTCALL, nullptr},
    {"grouped", fast(grouped), METH_FASTCALL, nullptr},
    {"grouped_backward", fast(grouped_backward), METH_FASTCALL, nullptr},
    {"lora", fast(lora), METH_FASTCALL, nullptr},
    {"has_tangent", fast(has_tangent), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", "Marshalling of the feed-forward and grouped calls.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `target` is what the module was built for; `key` also names the command that built it.
extern "C" __attribute__((visibility("default"))) PyObject* PyInit__calls(void) {
  PyObject* m = PyModule_Create(&g_module);
  if (m && (PyModule_AddStringConstant(m, "target", TG_CALLS_TARGET) < 0 ||
            PyModule_AddStringConstant(m, "key", TG_CALLS_KEY) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
