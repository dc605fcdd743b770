// The operators around the layer, called with torch tensors (module _calls).
//
// A single token's kernels take 3 to 5 us, so the host's side decides what a
// call costs.  In Python (attribute reads, struct packing, ctypes, torch.empty)
// a call took 8.1 to 10.2 us, here 4.7 to 5.5: the checks read the tensors'
// fields, and the results are allocated without Python's argument parsing.  The
// launch itself is 2.4 us of what remains.
//
// Checks of types, shapes, strides, devices and gradients stand here and raise ValueError;
// everything else (ranges, alignment, overlap) is the library's, whose status
// becomes the binding's error.  A call runs on its tensors' device and on that
// device's current stream, and makes its results there.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "nvfp4_moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;       // Nvfp4Error(status, message)
PyObject* g_raw_stream = nullptr;  // device index -> handle of its current stream
PyObject *g_weight, *g_bias, *g_desc;  // attribute names

[[noreturn]] void raised() {
  python_error e;
  e.persist();
  throw e;
}

struct Ref {  // an owned reference
  PyObject* p;
  explicit Ref(PyObject* p) : p(p) {
    if (!p) raised();
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_DECREF(p); }
};

int code_of(ScalarType t) {
  return t == ScalarType::BFloat16 ? MOE_BF16 : t == ScalarType::Half ? MOE_F16 : t == ScalarType::Float ? MOE_F32 : -1;
}

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_VALUE(t.is_cuda() && t.layout() == at::kStrided, name, " must be a CUDA tensor");
  // (the operators have no gradient: a result would leave the graph unnoticed)
  TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                    " requires a gradient, which this operator does not have (torch.no_grad() or detach it)");
  return t;
}

// A matrix of unit column stride, of bf16, f16 or f32 or of the given type.
const Tensor& matrix(PyObject* o, const char* name, ScalarType type = ScalarType::Undefined) {
  const Tensor& t = tensor(o, name);
  if (type == ScalarType::Undefined) {
    TORCH_CHECK_VALUE(code_of(t.scalar_type()) >= 0, name, " must be bfloat16, float16 or float32, got ", t.scalar_type());
  } else {
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  }
  TORCH_CHECK_VALUE(t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1), name, " must be a matrix with unit column stride");
  return t;
}

const Tensor& matrix_of(PyObject* o, const char* name, int64_t rows, int64_t cols, c10::Device device,
                        ScalarType type = ScalarType::Undefined) {
  const Tensor& t = matrix(o, name, type);
  TORCH_CHECK_VALUE(t.size(0) == rows && t.size(1) == cols && t.device() == device, name, " must be [", rows, ", ", cols,
                    "] on ", device, ", got ", t.sizes(), " on ", t.device());
  return t;
}

// The address of a contiguous vector of n values (NULL for None).
void* vector(PyObject* o, const char* name, int64_t n, ScalarType type, c10::Device device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.device() == device, name, " must be a tensor on ", device);
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && t.is_contiguous(), name,
                    " must be a contiguous ", type, " tensor of ", n, " values, got ", t.scalar_type(), " ", t.sizes());
  return t.data_ptr();
}

void* scales(PyObject* o, const char* name, int64_t n, c10::Device device) {
  TORCH_CHECK_VALUE(o != Py_None, name, " must be a tensor");
  return vector(o, name, n, ScalarType::Float, device);
}

// Elements between two rows (a single row's stride means nothing).
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// The same for 8-bit codes, whose rows start at multiples of 16 bytes.
int64_t code_stride(const Tensor& t, const char* name) {
  if (t.size(0) <= 1) return (t.size(1) + 15) / 16 * 16;
  TORCH_CHECK_VALUE(t.stride(0) % 16 == 0, name,
                    ": rows must start at multiples of 16 bytes, as int8_quantize_per_token lays them out");
  return t.stride(0);
}

Tensor empty(at::IntArrayRef shape, ScalarType type, c10::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

ScalarType type_of(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPDtype_Check(o) && code_of(reinterpret_cast<THPDtype*>(o)->scalar_type) >= 0, name,
                    " must be bfloat16, float16 or float32");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

float number(PyObject* o) {
  double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) raised();
  return static_cast<float>(v);
}

// The structure behind a Router or Norm (its attribute desc).
template <class S>
S structure(PyObject* o) {
  Ref desc(PyObject_GetAttr(o, g_desc));
  Py_buffer view;
  if (PyObject_GetBuffer(desc.p, &view, PyBUF_SIMPLE) != 0) raised();
  S s{};
  bool fits = view.len == sizeof(S);
  if (fits) std::memcpy(&s, view.buf, sizeof(S));
  PyBuffer_Release(&view);
  TORCH_CHECK_TYPE(fits, "a Router (for routing) or a Norm (for a norm) is expected");
  return s;
}

void* stream_of(c10::Device device) {
  Ref index(PyLong_FromLong(device.index())), s(PyObject_CallFunctionObjArgs(g_raw_stream, index.p, nullptr));
  void* p = PyLong_AsVoidPtr(s.p);
  if (!p && PyErr_Occurred()) raised();
  return p;
}

// Runs the library's function without the interpreter's lock; its status as an exception.
template <class F>
void call(F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = f();
  Py_END_ALLOW_THREADS;
  if (status == 0) return;
  Ref e(PyObject_CallFunction(g_error, "is", status, nvfp4_last_error()));
  PyErr_SetObject(g_error, e.p);
  raised();
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  Ref x(THPVariable_Wrap(a)), y(THPVariable_Wrap(b));
  return PyTuple_Pack(2, x.p, y.p);
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "takes ", want, " arguments, got ", n);
  TORCH_CHECK(g_error && g_raw_stream, "called before setup(error class, raw stream function)");
}

// (logits, top_k, router, bias, out)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const Tensor& logits = matrix(a[0], "logits");
  int64_t T = logits.size(0), E = logits.size(1);
  c10::Device device = logits.device();
  long k = PyLong_AsLong(a[1]);
  if (k == -1 && PyErr_Occurred()) raised();
  moe_router rule = structure<moe_router>(a[2]);
  auto* bias = static_cast<const float*>(vector(a[3], "bias", E, ScalarType::Float, device));
  int32_t top_k = static_cast<int32_t>(std::clamp(k, 0L, long{INT_MAX}));
  c10::DeviceGuard guard(device);
  Tensor ids, w;
  if (a[4] == Py_None) {
    int64_t made = std::min(top_k, 16);  // more are refused below
    ids = empty({T, made}, ScalarType::Int, device);
    w = empty({T, made}, ScalarType::Float, device);
  } else {
    TORCH_CHECK_VALUE(PyTuple_Check(a[4]) && PyTuple_GET_SIZE(a[4]) == 2, "out must be (ids, weights)");
    ids = matrix_of(PyTuple_GET_ITEM(a[4], 0), "ids", T, top_k, device, ScalarType::Int);
    w = matrix_of(PyTuple_GET_ITEM(a[4], 1), "weights", T, top_k, device, ScalarType::Float);
    TORCH_CHECK_VALUE(ids.is_contiguous() && w.is_contiguous(), "ids and weights must be contiguous");
  }
  void* stream = stream_of(device);
  call([&] {
    return moe_route(&rule, logits.data_ptr(), code_of(logits.scalar_type()), T, E, row_stride(logits), top_k, bias,
                     static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()), stream);
  });
  if (a[4] != Py_None) {
    Py_INCREF(a[4]);
    return a[4];
  }
  return pair(ids, w);
  END_HANDLE_TH_ERRORS
}

// A binding's norm with the weight and bias that it has now.
moe_norm norm_of(PyObject* o, int64_t cols, ScalarType type, c10::Device device) {
  moe_norm d = structure<moe_norm>(o);
  Ref w(PyObject_GetAttr(o, g_weight)), b(PyObject_GetAttr(o, g_bias));
  d.weight_dev = vector(w.p, "weight of a norm", cols, type, device);
  d.bias_dev = vector(b.p, "bias of a norm", cols, type, device);
  return d;
}

// (residual, y, before, after, gate, gate_sigmoid, res_scale, out_scale, residual_out, h_out)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  bool has_y = a[1] != Py_None, has_before = a[2] != Py_None, has_after = a[3] != Py_None, has_gate = a[4] != Py_None;
  const Tensor& residual = matrix(a[0], "residual");
  int64_t T = residual.size(0), H = residual.size(1);
  c10::Device device = residual.device();
  ScalarType rtype = residual.scalar_type(), type = rtype;

  moe_block_norm_args p{};
  p.rows = T;
  p.cols = H;
  p.residual_dtype = code_of(rtype);
  p.residual_dev = residual.data_ptr();
  p.ld_residual = row_stride(residual);
  if (has_y) {
    const Tensor& y = matrix_of(a[1], "y", T, H, device);
    type = y.scalar_type();
    p.y_dev = y.data_ptr();
    p.ld_y = row_stride(y);
  } else if (a[9] != Py_None) {
    type = matrix(a[9], "h_out").scalar_type();
  }
  p.dtype = code_of(type);
  if (has_gate) {
    const Tensor& gate = tensor(a[4], "gate");
    if (gate.dim() == 1) {
      p.gate_dev = vector(a[4], "gate", H, type, device);
      p.gate_cols = H;
    } else {
      matrix(a[4], "gate", type);
      TORCH_CHECK_VALUE(gate.device() == device && gate.size(0) == T && (gate.size(1) == 1 || gate.size(1) == H),
                        "gate must be [", H, "], [", T, ", 1] or [", T, ", ", H, "] on ", device, ", got ", gate.sizes(),
                        " on ", gate.device());
      p.gate_dev = gate.data_ptr();
      p.gate_cols = gate.size(1);
      p.ld_gate = row_stride(gate);
    }
  }
  int sigmoid = PyObject_IsTrue(a[5]);
  if (sigmoid < 0) raised();
  p.gate_sigmoid = sigmoid;
  p.res_scale = number(a[6]);
  p.out_scale = number(a[7]);
  moe_norm after, before;
  if (has_after) {
    after = norm_of(a[3], H, type, device);
    p.after = &after;
  }
  if (has_before) {
    before = norm_of(a[2], H, type, device);
    p.before = &before;
  }
  c10::DeviceGuard guard(device);
  Tensor r, h;
  if (a[8] != Py_None)
    r = matrix_of(a[8], "residual_out", T, H, device, rtype);
  else if (has_y || !has_before || p.res_scale != 1.0f)
    r = empty({T, H}, rtype, device);
  if (a[9] != Py_None) {
    TORCH_CHECK_VALUE(has_before, "h_out needs a norm (before)");
    h = matrix_of(a[9], "h_out", T, H, device, type);
  } else if (has_before) {
    h = empty({T, H}, type, device);
  }
  if (r.defined()) {
    p.residual_out_dev = r.data_ptr();
    p.ld_residual_out = row_stride(r);
  }
  if (h.defined()) {
    p.h_dev = h.data_ptr();
    p.ld_h = row_stride(h);
  }
  void* stream = stream_of(device);
  call([&] { return moe_block_norm(&p, stream); });
  return pair(r.defined() ? r : residual, h);  // an undefined tensor is None
  END_HANDLE_TH_ERRORS
}

// (x)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 1);
  const Tensor& x = matrix(a[0], "x");
  int64_t rows = x.size(0), cols = x.size(1), ld = (cols + 15) / 16 * 16;
  c10::Device device = x.device();
  c10::DeviceGuard guard(device);
  Tensor codes = empty({rows, ld}, ScalarType::Char, device), scale = empty({rows}, ScalarType::Float, device);
  void* stream = stream_of(device);
  call([&] {
    return int8_quantize_per_token(x.data_ptr(), code_of(x.scalar_type()), rows, cols, row_stride(x),
                                   static_cast<int8_t*>(codes.data_ptr()), ld, static_cast<float*>(scale.data_ptr()), stream);
  });
  return pair(ld != cols ? codes.narrow(1, 0, cols) : codes, scale);
  END_HANDLE_TH_ERRORS
}

Tensor product_out(PyObject* out, ScalarType type, int64_t M, int64_t N, c10::Device device) {
  return out == Py_None ? empty({M, N}, type, device) : matrix_of(out, "out", M, N, device);
}

// (codes, scale, w_codes, w_scale, bias, out_dtype, out)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor& codes = matrix(a[0], "codes", ScalarType::Char);
  int64_t M = codes.size(0), K = codes.size(1);
  c10::Device device = codes.device();
  const Tensor& w = matrix(a[2], "w_codes", ScalarType::Char);
  int64_t N = w.size(0);
  matrix_of(a[2], "w_codes", N, K, device, ScalarType::Char);
  auto* sa = static_cast<const float*>(scales(a[1], "scale", M, device));
  auto* sb = static_cast<const float*>(scales(a[3], "w_scale", N, device));
  auto* bias = static_cast<const float*>(vector(a[4], "bias", N, ScalarType::Float, device));
  int64_t lda = code_stride(codes, "codes"), ldb = code_stride(w, "w_codes");
  c10::DeviceGuard guard(device);
  Tensor out = product_out(a[6], a[6] == Py_None ? type_of(a[5], "out_dtype") : ScalarType::Undefined, M, N, device);
  void* stream = stream_of(device);
  call([&] {
    return int8_matmul(codes.data_ptr(), lda, sa, w.data_ptr(), ldb, sb, bias, M, N, K, out.data_ptr(),
                       code_of(out.scalar_type()), row_stride(out), stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (x, w_codes, w_scale, bias, out_dtype, out)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor& x = matrix(a[0], "x");
  int64_t M = x.size(0), K = x.size(1);
  c10::Device device = x.device();
  const Tensor& w = matrix(a[1], "w_codes", ScalarType::Char);
  int64_t N = w.size(0);
  matrix_of(a[1], "w_codes", N, K, device, ScalarType::Char);
  auto* sb = static_cast<const float*>(scales(a[2], "w_scale", N, device));
  auto* bias = static_cast<const float*>(vector(a[3], "bias", N, ScalarType::Float, device));
  int64_t ldb = code_stride(w, "w_codes"), bytes = 0;
  c10::DeviceGuard guard(device);
  Tensor out = product_out(a[5], a[4] == Py_None ? x.scalar_type() : type_of(a[4], "out_dtype"), M, N, device), work;
  call([&] { return int8_linear_workspace(M, K, &bytes); });
  if (bytes) work = empty({bytes}, ScalarType::Byte, device);
  void* stream = stream_of(device);
  call([&] {
    return int8_linear(x.data_ptr(), code_of(x.scalar_type()), row_stride(x), w.data_ptr(), ldb, sb, bias, M, N, K,
                       bytes ? work.data_ptr() : nullptr, bytes, out.data_ptr(), code_of(out.scalar_type()),
                       row_stride(out), stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (error class, raw_stream)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 2, "takes 2 arguments, got ", n);
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  g_error = a[0];
  g_raw_stream = a[1];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(route), CALL(block_norm), CALL(quantize), CALL(matmul),
                           CALL(linear), CALL(setup), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  g_weight = PyUnicode_InternFromString("weight");
  g_bias = PyUnicode_InternFromString("bias");
  g_desc = PyUnicode_InternFromString("desc");
  return g_weight && g_bias && g_desc ? PyModule_Create(&g_module) : nullptr;
}
