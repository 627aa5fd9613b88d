// Python module _skg_torch: the microscaled entry points of libskgemm.so, and those of a
// layer's projections in 16 bits, on torch tensors. It checks the arguments, allocates
// the outputs, and hands pointers, strides and the current stream to the C ABI; all
// arithmetic runs there. (A call of one token takes the GPU 3 to 4 us; the same
// marshalling in Python took 14 to 20 us.) Functions take their arguments by position,
// return the library's status (an int) when it refuses a call, and raise ValueError
// themselves.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "skgemm.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const char* kFormats[] = {"mxfp8", "mxfp4", "nvfp4"};

int format_of(PyObject* o) {
  if (PyUnicode_Check(o))
    for (int i = 0; i < 3; ++i)
      if (PyUnicode_CompareWithASCIIString(o, kFormats[i]) == 0) return i;
  PyObject* r = PyObject_Repr(o);
  const char* text = r ? PyUnicode_AsUTF8(r) : nullptr;
  const std::string what = std::string("unknown format ") + (text ? text : "?") +
                           ": one of mxfp8, mxfp4, nvfp4";
  Py_XDECREF(r);
  PyErr_Clear();
  refuse(what);
}

const at::Tensor& tensor_of(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor is wanted");
  return THPVariable_Unpack(o);
}

// skg_out_t (any = true) or skg_in_t of a tensor.
int type_of(const char* name, at::ScalarType t, bool any) {
  if (t == at::kHalf) return any ? SKG_OUT_F16 : SKG_IN_F16;
  if (t == at::kBFloat16) return any ? SKG_OUT_BF16 : SKG_IN_BF16;
  if (t == at::kFloat && any) return SKG_OUT_F32;
  refuse(std::string(name) + ": unsupported dtype " + c10::toString(t));
}

void on_device(const char* name, const at::Tensor& t, c10::Device d) {
  if (t.device() != d)
    refuse(std::string(name) + ": on " + t.device().str() + ", not on " + d.str());
}

// A row-major CUDA matrix; returns its row stride.
int64_t matrix(const char* name, const at::Tensor& t) {
  if (t.dim() != 2) refuse(std::string(name) + ": a matrix is wanted");
  if (!t.is_cuda()) refuse(std::string(name) + ": a CUDA tensor is wanted");
  if (t.size(1) > 1 && t.stride(1) != 1)
    refuse(std::string(name) + ": the last dimension must be contiguous");
  if (t.size(0) > 1) return t.stride(0);
  return t.size(1) > 0 ? t.size(1) : 1;
}

// The same with the type, shape and device of `like`.
int64_t matrix_like(const char* name, const at::Tensor& t, const at::Tensor& like) {
  const int64_t ld = matrix(name, t);
  if (t.size(0) != like.size(0) || t.size(1) != like.size(1))
    refuse(std::string(name) + ": a matrix of the other operands' shape is wanted");
  if (t.scalar_type() != like.scalar_type())
    refuse(std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()));
  on_device(name, t, like.device());
  return ld;
}

void* vector(const char* name, const at::Tensor& t, int64_t n, at::ScalarType type, c10::Device d) {
  if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type || (n > 1 && t.stride(0) != 1))
    refuse(std::string(name) + ": a contiguous vector of " + std::to_string(n) + " " +
           c10::toString(type) + " is wanted");
  on_device(name, t, d);
  return t.data_ptr();
}

// A tensor scale (None: NULL).
const float* scalar(const char* name, PyObject* o, c10::Device d) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor_of(name, o);
  if (t.numel() != 1 || t.scalar_type() != at::kFloat)
    refuse(std::string(name) + ": one float32 on the device is wanted");
  on_device(name, t, d);
  return (const float*)t.data_ptr();
}

const float* tensor_scale(PyObject* o, int fmt, c10::Device d) {
  if (o != Py_None && fmt != SKG_NVFP4) refuse("tensor_scale belongs to nvfp4");
  return scalar("tensor_scale", o, d);
}

void* stream_of(c10::Device d) {
  return (void*)c10::cuda::getCurrentCUDAStream(d.index()).stream();
}

// An uninitialised contiguous CUDA tensor, past the dispatcher.
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device d) {
  return at::detail::empty_cuda(sizes, type, d, std::nullopt);
}

bool flag(const char* name, PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + ": a truth value is wanted");
  }
  return v == 1;
}

struct Quantized {
  at::Tensor codes, scales;
  int64_t ldq;
  Quantized(int64_t rows, int64_t k, int fmt, c10::Device d)
      : ldq(skg_mx_codes_ld(k, fmt)) {
    codes = empty({rows, ldq}, at::kByte, d);
    scales = empty({(int64_t)skg_mx_scales_size(rows, k, fmt)}, at::kByte, d);
  }
};

// A given output is written: autograd sees it changed, as after any operation in place.
PyObject* written(const at::Tensor& out) {
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
  return THPVariable_Wrap(out);
}

PyObject* wrap_or_none(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, wrap_or_none(t));
  return out;
}

void want(Py_ssize_t n, Py_ssize_t count) {
  if (n != count) refuse(std::to_string(count) + " arguments are wanted");
}

// quantize(x, format, transpose, tensor_scale, values) -> (codes, scales, values)
PyObject* quantize(PyObject* const* a, Py_ssize_t n) {
  want(n, 5);
  const int fmt = format_of(a[1]);
  const at::Tensor& x = tensor_of("x", a[0]);
  const int type = type_of("x", x.scalar_type(), true);
  const int64_t ldx = matrix("x", x);
  const bool tr = flag("transpose", a[2]), values = flag("values", a[4]);
  const c10::cuda::CUDAGuard guard(x.device());
  const float* g = tensor_scale(a[3], fmt, x.device());
  const int64_t rows = x.size(tr ? 1 : 0), k = x.size(tr ? 0 : 1);
  Quantized q(rows, k, fmt, x.device());
  at::Tensor v;
  if (values) v = empty({rows, k}, x.scalar_type(), x.device());
  const int st = skg_mx_quantize(rows, k, x.data_ptr(), ldx, type, tr ? 1 : 0, fmt, g,
                                 q.codes.data_ptr(), q.ldq, q.scales.data_ptr(),
                                 values ? v.data_ptr() : nullptr, k, stream_of(x.device()));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({q.codes, q.scales, v});
}

// quantize_both(x, format, tensor_scale) -> (codes, scales, codes_t, scales_t)
PyObject* quantize_both(PyObject* const* a, Py_ssize_t n) {
  want(n, 3);
  const int fmt = format_of(a[1]);
  const at::Tensor& x = tensor_of("x", a[0]);
  const int type = type_of("x", x.scalar_type(), true);
  const int64_t ldx = matrix("x", x);
  const c10::cuda::CUDAGuard guard(x.device());
  const float* g = tensor_scale(a[2], fmt, x.device());
  const int64_t rows = x.size(0), cols = x.size(1);
  Quantized q(rows, cols, fmt, x.device()), t(cols, rows, fmt, x.device());
  const int st = skg_mx_quantize_both(rows, cols, x.data_ptr(), ldx, type, fmt, g,
                                      q.codes.data_ptr(), q.ldq, q.scales.data_ptr(),
                                      t.codes.data_ptr(), t.ldq, t.scales.data_ptr(),
                                      stream_of(x.device()));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({q.codes, q.scales, t.codes, t.scales});
}

// rmsnorm(x, weight, eps, residual, format, tensor_scale) -> (codes, scales, sum, rstd)
PyObject* rmsnorm(PyObject* const* a, Py_ssize_t n) {
  want(n, 6);
  const int fmt = format_of(a[4]);
  const at::Tensor& x = tensor_of("x", a[0]);
  const int type = type_of("x", x.scalar_type(), false);
  const int64_t ldx = matrix("x", x);
  const int64_t rows = x.size(0), cols = x.size(1);
  const c10::Device d = x.device();
  const c10::cuda::CUDAGuard guard(d);
  const void* w = vector("weight", tensor_of("weight", a[1]), cols, x.scalar_type(), d);
  const double eps = PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const float* g = tensor_scale(a[5], fmt, d);
  const void* r = nullptr;
  int64_t ldr = 0;
  at::Tensor sum;
  if (a[3] != Py_None) {
    const at::Tensor& res = tensor_of("residual", a[3]);
    ldr = matrix_like("residual", res, x);
    r = res.data_ptr();
    sum = empty({rows, cols}, x.scalar_type(), d);
  }
  Quantized q(rows, cols, fmt, d);
  at::Tensor rstd = empty({rows}, at::kFloat, d);
  const int st = skg_rmsnorm_mx(rows, cols, x.data_ptr(), ldx, r, ldr, w, type, (float)eps,
                                sum.defined() ? sum.data_ptr() : nullptr, cols,
                                (float*)rstd.data_ptr(), fmt, g, q.codes.data_ptr(), q.ldq,
                                q.scales.data_ptr(), stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({q.codes, q.scales, sum, rstd});
}

// rmsnorm_backward(dy, h, weight, rstd, dresidual) -> (dx, dweight)
PyObject* rmsnorm_backward(PyObject* const* a, Py_ssize_t n) {
  want(n, 5);
  const at::Tensor& dy = tensor_of("dy", a[0]);
  const int type = type_of("dy", dy.scalar_type(), false);
  const int64_t ldy = matrix("dy", dy);
  const int64_t rows = dy.size(0), cols = dy.size(1);
  const c10::Device d = dy.device();
  const c10::cuda::CUDAGuard guard(d);
  const at::Tensor& h = tensor_of("h", a[1]);
  const int64_t ldh = matrix_like("h", h, dy);
  const void* w = vector("weight", tensor_of("weight", a[2]), cols, dy.scalar_type(), d);
  const void* rstd = vector("rstd", tensor_of("rstd", a[3]), rows, at::kFloat, d);
  const void* dr = nullptr;
  int64_t ldr = 0;
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor_of("dresidual", a[4]);
    ldr = matrix_like("dresidual", t, dy);
    dr = t.data_ptr();
  }
  const size_t bytes = skg_workspace_size_rmsnorm_backward(rows, cols);
  at::Tensor dx = empty({rows, cols}, dy.scalar_type(), d);
  at::Tensor dw = empty({cols}, at::kFloat, d);
  at::Tensor ws = empty({(int64_t)bytes}, at::kByte, d);
  const int st = skg_rmsnorm_backward(rows, cols, dy.data_ptr(), ldy, h.data_ptr(), ldh, w,
                                      (const float*)rstd, dr, ldr, type, dx.data_ptr(), cols,
                                      (float*)dw.data_ptr(), ws.data_ptr(), bytes, stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({dx, dw});
}

// A Matrix: (format, rows, k, codes, scales, tensor_scale).
struct Operand {
  int fmt;
  int64_t rows, k, ld;
  const at::Tensor *codes, *scales;
  const float* g;
};

Operand operand(const std::string& name, PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) refuse(name + ": a Matrix is wanted");
  Operand q;
  q.fmt = format_of(PyTuple_GET_ITEM(o, 0));
  q.rows = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1));
  q.k = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name + ": rows and k are integers");
  }
  q.codes = &tensor_of("codes", PyTuple_GET_ITEM(o, 3));
  q.scales = &tensor_of("scales", PyTuple_GET_ITEM(o, 4));
  const at::Tensor &c = *q.codes, &s = *q.scales;
  if (q.rows < 0 || q.k < 0 || c.scalar_type() != at::kByte || s.scalar_type() != at::kByte ||
      c.dim() != 2 || c.size(0) != q.rows || c.size(1) < skg_mx_codes_ld(q.k, q.fmt) ||
      (c.size(1) > 1 && c.stride(1) != 1) || !c.is_cuda() || !s.is_contiguous() ||
      s.numel() < (int64_t)skg_mx_scales_size(q.rows, q.k, q.fmt))
    refuse(name + ": codes or scales are not those of a " + std::to_string(q.rows) + " x " +
           std::to_string(q.k) + " " + kFormats[q.fmt] + " matrix on a CUDA device");
  on_device((name + ".scales").c_str(), s, c.device());
  q.ld = q.rows > 1 ? c.stride(0) : c.size(1);
  q.g = scalar((name + ".tensor_scale").c_str(), PyTuple_GET_ITEM(o, 5), c.device());
  return q;
}

// matmul(a, b, out or None, out_dtype, alpha, beta, workspace) -> out
PyObject* matmul(PyObject* const* v, Py_ssize_t n) {
  want(n, 7);
  const Operand a = operand("a", v[0]), b = operand("b", v[1]);
  if (a.fmt != b.fmt)
    refuse(std::string("b: ") + kFormats[b.fmt] + ", the other operand is " + kFormats[a.fmt]);
  if (a.k != b.k)
    refuse("a has rows of " + std::to_string(a.k) + " elements, b of " + std::to_string(b.k));
  const c10::Device d = a.codes->device();
  on_device("b", *b.codes, d);
  const c10::cuda::CUDAGuard guard(d);
  const double alpha = PyFloat_AsDouble(v[4]), beta = PyFloat_AsDouble(v[5]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor out;
  int64_t ldc = b.rows;
  if (v[2] == Py_None) {
    if (beta != 0.0) refuse("beta is for a given out");
    if (!THPDtype_Check(v[3])) refuse("out_dtype: a dtype is wanted");
    const at::ScalarType t = reinterpret_cast<THPDtype*>(v[3])->scalar_type;
    type_of("out_dtype", t, true);
    out = empty({a.rows, b.rows}, t, d);
  } else {
    out = tensor_of("out", v[2]);
    ldc = matrix("out", out);
    if (out.size(0) != a.rows || out.size(1) != b.rows)
      refuse("out: a matrix of shape (" + std::to_string(a.rows) + ", " + std::to_string(b.rows) +
             ") is wanted");
    on_device("out", out, d);
  }
  const at::Tensor& ws = tensor_of("workspace", v[6]);
  on_device("workspace", ws, d);
  const int st = skg_gemm_mx(a.rows, b.rows, a.k, (float)alpha, a.codes->data_ptr(), a.ld,
                             a.scales->data_ptr(), a.g, b.codes->data_ptr(), b.ld,
                             b.scales->data_ptr(), b.g, (float)beta, out.data_ptr(), ldc, a.fmt,
                             type_of("out", out.scalar_type(), true), ws.data_ptr(),
                             (size_t)ws.nbytes(), stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : written(out);
}

// ------------------------------------------------------------------ a layer's projections
const char* kActivations[] = {"silu", "gelu", "gelu_tanh", "relu"};

int activation_of(PyObject* o) {
  if (PyUnicode_Check(o))
    for (int i = 0; i < 4; ++i)
      if (PyUnicode_CompareWithASCIIString(o, kActivations[i]) == 0) return i;
  refuse("unknown activation: one of silu, gelu, gelu_tanh, relu");
}

// A 16-bit matrix (rows, cols) of x's type and device (cols < 0: any); returns its row stride.
int64_t operand_like(const char* name, const at::Tensor& t, int64_t rows, int64_t cols,
                     const at::Tensor& x) {
  const int64_t ld = matrix(name, t);
  if (t.size(0) != rows || (cols >= 0 && t.size(1) != cols))
    refuse(std::string(name) + ": a matrix of " + std::to_string(rows) + " x " +
           (cols < 0 ? "?" : std::to_string(cols)) + " is wanted");
  if (t.scalar_type() != x.scalar_type())
    refuse(std::string(name) + ": " + c10::toString(t.scalar_type()) + ", the other operands are " +
           c10::toString(x.scalar_type()));
  on_device(name, t, x.device());
  return ld;
}

// An uninitialised matrix whose rows start on 16-byte boundaries.
at::Tensor padded(int64_t rows, int64_t cols, const at::Tensor& x) {
  const int64_t ld = (cols + 7) / 8 * 8;
  at::Tensor t = empty({rows, ld}, x.scalar_type(), x.device());
  return ld == cols ? t : t.narrow(1, 0, cols);
}

int64_t ld_of(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

at::Tensor scratch_of(size_t bytes, c10::Device d) {
  return empty({(int64_t)(bytes ? bytes : 1)}, at::kByte, d);
}

// One matrix of a stack (count, rows, cols): its row and matrix strides.
void stack_like(const char* name, const at::Tensor& t, int64_t count, int64_t rows, int64_t cols,
                const at::Tensor& x, int64_t* ld, int64_t* stride) {
  if (t.dim() != 3 || t.size(0) != count || t.size(1) != rows || t.size(2) != cols)
    refuse(std::string(name) + ": a stack of " + std::to_string(count) + " x " +
           std::to_string(rows) + " x " + std::to_string(cols) + " is wanted");
  if (t.scalar_type() != x.scalar_type())
    refuse(std::string(name) + ": " + c10::toString(t.scalar_type()) + ", x is " +
           c10::toString(x.scalar_type()));
  on_device(name, t, x.device());
  if (cols > 1 && t.stride(2) != 1)
    refuse(std::string(name) + ": the last dimension must be contiguous");
  *ld = rows > 1 ? t.stride(1) : cols;
  *stride = count > 1 ? t.stride(0) : rows * cols;
}

// linear(x, w, (a, b, scale) or None, index, out or None, workspace) -> y
PyObject* linear(PyObject* const* v, Py_ssize_t n) {
  want(n, 6);
  const at::Tensor& x = tensor_of("x", v[0]);
  const int type = type_of("x", x.scalar_type(), false);
  const int64_t ldx = matrix("x", x);
  const int64_t m = x.size(0), k = x.size(1);
  const c10::Device d = x.device();
  const c10::cuda::CUDAGuard guard(d);
  const at::Tensor& w = tensor_of("w", v[1]);
  if (w.dim() != 2) refuse("w: a matrix is wanted");
  const int64_t ldw = operand_like("w", w, w.size(0), k, x), rows = w.size(0);
  skg_adapters_t ad = {};
  const bool adapted = v[2] != Py_None;
  if (!adapted && v[3] != Py_None) refuse("index belongs to adapters");
  if (adapted) {
    if (!PyTuple_Check(v[2]) || PyTuple_GET_SIZE(v[2]) != 3) refuse("adapters: Adapters are wanted");
    const at::Tensor& a = tensor_of("adapters.down", PyTuple_GET_ITEM(v[2], 0));
    const at::Tensor& b = tensor_of("adapters.up", PyTuple_GET_ITEM(v[2], 1));
    if (a.dim() != 3) refuse("adapters.down: a stack of matrices is wanted");
    if (a.size(0) > INT32_MAX || a.size(1) > INT32_MAX) refuse("adapters.down: too many");
    ad.count = (int32_t)a.size(0);
    ad.rank = (int32_t)a.size(1);
    stack_like("adapters.down", a, ad.count, ad.rank, k, x, &ad.ld_down, &ad.stride_down);
    stack_like("adapters.up", b, ad.count, rows, ad.rank, x, &ad.ld_up, &ad.stride_up);
    ad.down = a.data_ptr();
    ad.up = b.data_ptr();
    ad.index = (const int32_t*)vector("index", tensor_of("index", v[3]), m, at::kInt, d);
    PyObject* scale = PyTuple_GET_ITEM(v[2], 2);
    if (scale != Py_None)
      ad.scale = (const float*)vector("adapters.scale", tensor_of("adapters.scale", scale),
                                      ad.count, at::kFloat, d);
  }
  const at::Tensor& ws = tensor_of("workspace", v[5]);
  on_device("workspace", ws, d);
  at::Tensor out;
  int64_t ldo;
  if (v[4] == Py_None) {
    out = padded(m, rows, x);
    ldo = ld_of(out);
  } else {
    out = tensor_of("out", v[4]);
    ldo = operand_like("out", out, m, rows, x);
  }
  const size_t bytes = adapted ? skg_scratch_size_linear(m, ad.rank) : 0;
  at::Tensor scratch;
  if (bytes) scratch = scratch_of(bytes, d);
  const int st = skg_linear(m, rows, k, x.data_ptr(), ldx, w.data_ptr(), ldw,
                            adapted ? &ad : nullptr, out.data_ptr(), ldo, type, ws.data_ptr(),
                            (size_t)ws.nbytes(), bytes ? scratch.data_ptr() : nullptr, bytes,
                            stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : written(out);
}

// Rows of one projection of w_in (2 hidden, k).
int64_t hidden_of(const at::Tensor& w, int64_t k) {
  if (w.dim() != 2 || w.size(0) % 2 || w.size(1) != k)
    refuse("w_in: a matrix of 2 hidden x " + std::to_string(k) + " is wanted");
  return w.size(0) / 2;
}

// gated(x, w_in, activation, save, workspace) -> (h, pre or None)
PyObject* gated(PyObject* const* v, Py_ssize_t n) {
  want(n, 5);
  const at::Tensor& x = tensor_of("x", v[0]);
  const int type = type_of("x", x.scalar_type(), false);
  const int64_t ldx = matrix("x", x);
  const int64_t m = x.size(0), k = x.size(1);
  const c10::Device d = x.device();
  const c10::cuda::CUDAGuard guard(d);
  const at::Tensor& w = tensor_of("w_in", v[1]);
  const int64_t f = hidden_of(w, k), ldw = operand_like("w_in", w, 2 * f, k, x);
  const int act = activation_of(v[2]);
  const bool save = flag("save", v[3]);
  const at::Tensor& ws = tensor_of("workspace", v[4]);
  on_device("workspace", ws, d);
  at::Tensor h = padded(m, f, x), pre;
  if (save) pre = padded(m, 2 * f, x);
  const int st = skg_gated(m, f, k, x.data_ptr(), ldx, w.data_ptr(), ldw, act, h.data_ptr(),
                           ld_of(h), save ? pre.data_ptr() : nullptr, save ? ld_of(pre) : 0, type,
                           ws.data_ptr(), (size_t)ws.nbytes(), stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({h, pre});
}

// gated_backward(dh, x, w_in, pre, activation, workspace) -> (dx, dw_in)
PyObject* gated_backward(PyObject* const* v, Py_ssize_t n) {
  want(n, 6);
  const at::Tensor& x = tensor_of("x", v[1]);
  const int type = type_of("x", x.scalar_type(), false);
  const int64_t ldx = matrix("x", x);
  const int64_t m = x.size(0), k = x.size(1);
  const c10::Device d = x.device();
  const c10::cuda::CUDAGuard guard(d);
  const at::Tensor &dh = tensor_of("dh", v[0]), &w = tensor_of("w_in", v[2]),
                   &pre = tensor_of("pre", v[3]);
  const int64_t f = hidden_of(w, k), ldw = operand_like("w_in", w, 2 * f, k, x),
                lddh = operand_like("dh", dh, m, f, x), ldp = operand_like("pre", pre, m, 2 * f, x);
  const int act = activation_of(v[4]);
  const at::Tensor& ws = tensor_of("workspace", v[5]);
  on_device("workspace", ws, d);
  at::Tensor dx = padded(m, k, x), dw = padded(2 * f, k, x);
  const size_t bytes = skg_scratch_size_gated_backward(m, f);
  at::Tensor scratch = scratch_of(bytes, d);
  const int st = skg_gated_backward(m, f, k, dh.data_ptr(), lddh, x.data_ptr(), ldx, w.data_ptr(),
                                    ldw, pre.data_ptr(), ldp, act, dx.data_ptr(), ld_of(dx),
                                    dw.data_ptr(), ld_of(dw), type, ws.data_ptr(),
                                    (size_t)ws.nbytes(), scratch.data_ptr(), bytes, stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({dx, dw});
}

// feed_forward_backward(dy, x, w_in, w_out, pre, activation, workspace) -> (dx, dw_in, dw_out)
PyObject* feed_forward_backward(PyObject* const* v, Py_ssize_t n) {
  want(n, 7);
  const at::Tensor& x = tensor_of("x", v[1]);
  const int type = type_of("x", x.scalar_type(), false);
  const int64_t ldx = matrix("x", x);
  const int64_t m = x.size(0), k = x.size(1);
  const c10::Device d = x.device();
  const c10::cuda::CUDAGuard guard(d);
  const at::Tensor &dy = tensor_of("dy", v[0]), &wi = tensor_of("w_in", v[2]),
                   &wo = tensor_of("w_out", v[3]), &pre = tensor_of("pre", v[4]);
  const int64_t f = hidden_of(wi, k), ldwi = operand_like("w_in", wi, 2 * f, k, x),
                ldwo = operand_like("w_out", wo, k, f, x), lddy = operand_like("dy", dy, m, k, x),
                ldp = operand_like("pre", pre, m, 2 * f, x);
  const int act = activation_of(v[5]);
  const at::Tensor& ws = tensor_of("workspace", v[6]);
  on_device("workspace", ws, d);
  at::Tensor dx = padded(m, k, x), dwi = padded(2 * f, k, x), dwo = padded(k, f, x);
  const size_t bytes = skg_scratch_size_feed_forward_backward(m, f);
  at::Tensor scratch = scratch_of(bytes, d);
  const int st = skg_feed_forward_backward(
      m, f, k, dy.data_ptr(), lddy, x.data_ptr(), ldx, wi.data_ptr(), ldwi, wo.data_ptr(), ldwo,
      pre.data_ptr(), ldp, act, dx.data_ptr(), ld_of(dx), dwi.data_ptr(), ld_of(dwi),
      dwo.data_ptr(), ld_of(dwo), type, ws.data_ptr(), (size_t)ws.nbytes(), scratch.data_ptr(),
      bytes, stream_of(d));
  return st != SKG_OK ? PyLong_FromLong(st) : tuple_of({dx, dwi, dwo});
}

// No C++ exception crosses into the interpreter.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define SKG_ENTRY(name) \
  {#name, (PyCFunction)(void (*)(void))entry<name>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {SKG_ENTRY(quantize), SKG_ENTRY(quantize_both), SKG_ENTRY(rmsnorm),
                          SKG_ENTRY(rmsnorm_backward), SKG_ENTRY(matmul),
                          SKG_ENTRY(linear), SKG_ENTRY(gated), SKG_ENTRY(gated_backward),
                          SKG_ENTRY(feed_forward_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_skg_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__skg_torch(void) { return PyModule_Create(&kModule); }
