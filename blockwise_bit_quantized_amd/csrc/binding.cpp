// binding.cpp -- the host side of the torch binding of include/mnb_ops.h (module _mnb_ops): checks
// of arguments, output and scratch allocation, and the C call, in one native call.
//
// A single-token call is bound by the host: a launch takes about 3.2 us, and the same
// steps in Python (attribute reads, allocations, ctypes) took 4 to 10 us on top of it where
// these take 2 to 3.  The module holds no state but the addresses of the C functions, which
// `bind` receives once; every function takes the stream handle first.  Forward only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <string>

#include "mnb_ops.h"

namespace {

struct {
  decltype(&mnb_mx_quantize) quantize;
  decltype(&mnb_mx_dequantize) dequantize;
  decltype(&mnb_mx_matmul) matmul;
  decltype(&mnb_rmsnorm) rmsnorm;
  decltype(&mnb_logprobs) logprobs;
  decltype(&mnb_logprobs_workspace_bytes) logprobs_ws;
  decltype(&mnb_status_string) status_string;
} c;

// A Python exception on its way out of a check.
struct Raised {};

[[noreturn]] void fail(PyObject *type, const char *format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised();
}

std::string shape_of(const at::Tensor &t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

at::Tensor tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
at::Tensor maybe_tensor(PyObject *o, const char *name) { return o == Py_None ? at::Tensor() : tensor(o, name); }
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
void *pointer(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}
PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
void *data(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return MNB_F16;
    case at::kBFloat16: return MNB_BF16;
    case at::kFloat: return MNB_F32;
    default: return -1;
  }
}
int float_type(const at::Tensor &t, const char *name, bool f32) {
  const int code = type_code(t.scalar_type());
  if (code < 0 || (code == MNB_F32 && !f32))
    fail(PyExc_TypeError, "%s must be float16%s, got %s", name, f32 ? ", bfloat16 or float32" : " or bfloat16",
         at::toString(t.scalar_type()));
  return code;
}

// The row distance of a 2-D tensor whose rows are contiguous and do not overlap.
int64_t row_distance(const at::Tensor &t, const char *name) {
  if (t.dim() != 2) fail(PyExc_ValueError, "%s must be 2-D, got shape %s", name, shape_of(t).c_str());
  const int64_t n = t.size(0), k = t.size(1);
  if (k > 1 && t.stride(1) != 1) fail(PyExc_ValueError, "the rows of %s must be contiguous", name);
  if (n <= 1) return k ? k : 1;
  if (t.stride(0) < k) fail(PyExc_ValueError, "the rows of %s must not overlap", name);
  return t.stride(0);
}
// ... of a tensor that has to match another's type, shape and device
int64_t row_distance_beside(const at::Tensor &t, const char *name, at::ScalarType type, int64_t n, int64_t k, at::Device dev) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != k)
    fail(PyExc_ValueError, "%s has shape %s, expected [%lld, %lld]", name, shape_of(t).c_str(), (long long)n, (long long)k);
  if (t.device() != dev)
    fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
  return row_distance(t, name);
}
void vector(const at::Tensor &t, const char *name, at::ScalarType type, int64_t n, at::Device dev) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    fail(PyExc_ValueError, "%s must be a contiguous [%lld], got shape %s", name, (long long)n, shape_of(t).c_str());
  if (t.device() != dev)
    fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
}
void blocks(int64_t K, const char *name) {
  if (K % 32) fail(PyExc_ValueError, "the last axis of %s must be a multiple of 32, got %lld", name, (long long)K);
}
void on_gpu(const at::Tensor &t) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "tensors must be on a GPU, got %s", t.device().str().c_str());
}
// the C calls take int sizes
int size(int64_t v) {
  if (v > INT32_MAX) fail(PyExc_ValueError, "a dimension of %lld is too large", (long long)v);
  return (int)v;
}
void check(int status) {
  if (status != MNB_OK) fail(PyExc_RuntimeError, "%s", c.status_string(status));
}

// a caller's tensor that the call wrote into: its version tells a graph that saved it
void written(const at::Tensor &t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

at::Tensor empty(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type));
}

// a new MX tensor on the device of `like`
struct Mx {
  at::Tensor codes, scales;
  int64_t ldc = 0, lds = 0;
  Mx(const at::Tensor &like, int64_t rows, int64_t K, int fmt) {
    if (fmt != MNB_MX_FP4 && fmt != MNB_MX_FP8) fail(PyExc_ValueError, "unknown MX format %d", fmt);
    ldc = fmt == MNB_MX_FP4 ? K / 2 : K;
    lds = (K + 511) / 512 * 16;
    codes = empty({rows, ldc}, like, at::kByte);
    scales = empty({rows, lds}, like, at::kByte);
    if (lds != K / 32) scales = scales.as_strided({rows, K / 32}, {lds, 1});
  }
};

// quantize(stream, x, fmt) -> (codes, scales, ldc, lds, rows, K)
PyObject *quantize(PyObject *const *a) {
  const at::Tensor x = tensor(a[1], "x");
  const int code = float_type(x, "x", true), fmt = (int)integer(a[2]);
  const int64_t ldx = row_distance(x, "x"), M = x.size(0), K = x.size(1);
  blocks(K, "x");
  const Mx q(x, M, K, fmt);
  on_gpu(x);
  check(c.quantize(data(x), code, size(M), size(K), ldx, fmt, data(q.codes), q.ldc, data(q.scales), q.lds, pointer(a[0])));
  return Py_BuildValue("NNLLLL", wrap(q.codes), wrap(q.scales), (long long)q.ldc, (long long)q.lds, (long long)M, (long long)K);
}

// dequantize(stream, codes, scales, fmt, rows, K, ldc, lds, dtype, out) -> y
PyObject *dequantize(PyObject *const *a) {
  const at::Tensor codes = tensor(a[1], "codes"), scales = tensor(a[2], "scales");
  at::Tensor y = maybe_tensor(a[9], "out");
  if (!THPDtype_Check(a[8])) fail(PyExc_TypeError, "dtype must be a torch dtype");
  const at::ScalarType type = reinterpret_cast<THPDtype *>(a[8])->scalar_type;
  const int fmt = (int)integer(a[3]);
  const int64_t M = integer(a[4]), K = integer(a[5]);
  if (type_code(type) < 0) fail(PyExc_TypeError, "the output must be float16, bfloat16 or float32");
  int64_t ldy = K;
  if (y.defined()) ldy = row_distance_beside(y, "out", type, M, K, codes.device());
  else y = empty({M, K}, codes, type);
  on_gpu(codes);
  check(c.dequantize(data(codes), integer(a[6]), data(scales), integer(a[7]), fmt, size(M), size(K), data(y), type_code(type), ldy,
                     pointer(a[0])));
  if (a[9] != Py_None) written(y);
  return wrap(y);
}

// matmul(stream, codes, scales, fmt, rows, K, ldc, lds, wq, sc, N, weight_K, bias, dtype, out) -> y
PyObject *matmul(PyObject *const *a) {
  const at::Tensor codes = tensor(a[1], "codes"), scales = tensor(a[2], "scales"), wq = tensor(a[8], "wq"), sc = tensor(a[9], "sc"),
                   bias = maybe_tensor(a[12], "bias");
  at::Tensor y = maybe_tensor(a[14], "out");
  const int fmt = (int)integer(a[3]);
  const int64_t M = integer(a[4]), K = integer(a[5]), N = integer(a[10]), wK = integer(a[11]);
  if (!THPDtype_Check(a[13])) fail(PyExc_TypeError, "dtype must be a torch dtype");
  const at::ScalarType type = reinterpret_cast<THPDtype *>(a[13])->scalar_type;
  const int code = type_code(type);
  if (code != MNB_F16 && code != MNB_BF16)
    fail(PyExc_TypeError, "the output must be float16 or bfloat16, got %s", at::toString(type));
  if (K != wK) fail(PyExc_ValueError, "x has K=%lld, weight has K=%lld", (long long)K, (long long)wK);
  if (wq.device() != codes.device())
    fail(PyExc_ValueError, "the weight is on %s, expected %s", wq.device().str().c_str(), codes.device().str().c_str());
  if (!y.defined()) y = empty({M, N}, codes, type);
  else if (y.scalar_type() != type || y.dim() != 2 || y.size(0) != M || y.size(1) != N || !y.is_contiguous() ||
           y.device() != codes.device())
    fail(PyExc_ValueError, "out must be a contiguous %s [%lld, %lld] on %s", at::toString(type), (long long)M, (long long)N,
         codes.device().str().c_str());
  if (bias.defined()) vector(bias, "bias", type, N, codes.device());
  on_gpu(codes);
  check(c.matmul(data(codes), integer(a[6]), data(scales), integer(a[7]), fmt, data(wq), data(sc), data(bias), data(y), code, size(M),
                 size(N), size(K), pointer(a[0])));
  if (a[14] != Py_None) written(y);
  return wrap(y);
}

// rmsnorm(stream, x, weight, eps, residual, fmt or None, keep16, out, hidden)
//   -> (y, hidden, codes, scales, ldc, lds, rows, K)
PyObject *rmsnorm(PyObject *const *a) {
  const at::Tensor x = tensor(a[1], "x"), weight = tensor(a[2], "weight"), residual = maybe_tensor(a[4], "residual");
  at::Tensor y = maybe_tensor(a[7], "out"), hidden = maybe_tensor(a[8], "hidden");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const int code = float_type(x, "x", false);
  const int64_t ldx = row_distance(x, "x"), M = x.size(0), K = x.size(1);
  const at::ScalarType type = x.scalar_type();
  vector(weight, "weight", type, K, x.device());
  int64_t ldr = 0, ldh = 0, ldy = 0;
  if (residual.defined()) {
    ldr = row_distance_beside(residual, "residual", type, M, K, x.device());
    if (hidden.defined()) ldh = row_distance_beside(hidden, "hidden", type, M, K, x.device());
    else hidden = empty({M, ldh = K}, x, type);
  } else if (hidden.defined()) {
    fail(PyExc_ValueError, "hidden needs a residual");
  }
  const bool mx = a[5] != Py_None, keep16 = !mx || truth(a[6]);
  if (mx) blocks(K, "x");
  if (y.defined()) ldy = row_distance_beside(y, "out", type, M, K, x.device());
  else if (keep16) y = empty({M, ldy = K}, x, type);
  at::Tensor codes, scales;
  int64_t ldc = 0, lds = 0;
  int fmt = 0;
  if (mx) {
    fmt = (int)integer(a[5]);
    Mx q(x, M, K, fmt);
    codes = q.codes;
    scales = q.scales;
    ldc = q.ldc;
    lds = q.lds;
  }
  on_gpu(x);
  check(c.rmsnorm(data(x), ldx, data(residual), ldr, data(weight), (float)eps, code, size(M), size(K), data(hidden), ldh, data(y), ldy,
                  fmt, data(codes), ldc, data(scales), lds, pointer(a[0])));
  if (a[7] != Py_None) written(y);
  if (a[8] != Py_None) written(hidden);
  return Py_BuildValue("NNNNLLLL", wrap(y), wrap(hidden), wrap(codes), wrap(scales), (long long)ldc, (long long)lds, (long long)M,
                       (long long)K);
}

// logprobs(stream, logits, tokens, top) -> (logprob, entropy, top_logprobs, top_tokens)
PyObject *logprobs(PyObject *const *a) {
  const at::Tensor x = tensor(a[1], "logits"), tokens = maybe_tensor(a[2], "tokens");
  const int64_t top = integer(a[3]);
  const int code = float_type(x, "logits", true);
  const int64_t ldl = row_distance(x, "logits"), M = x.size(0), V = x.size(1);
  const int64_t most = V < MNB_LOGPROBS_MAX_TOP ? V : MNB_LOGPROBS_MAX_TOP;
  if (top < 0 || top > most) fail(PyExc_ValueError, "top must be from 0 to %lld, got %lld", (long long)most, (long long)top);
  if (V == 0 && M > 0) fail(PyExc_ValueError, "logits have no columns");
  at::Tensor lp, tl, tt, ws;
  if (tokens.defined()) {
    vector(tokens, "tokens", at::kLong, M, x.device());
    lp = empty({M}, x, at::kFloat);
  }
  const at::Tensor ent = empty({M}, x, at::kFloat);
  if (top) {
    tl = empty({M, top}, x, at::kFloat);
    tt = empty({M, top}, x, at::kLong);
  }
  on_gpu(x);
  const size_t need = c.logprobs_ws(size(M), size(V), code, (int)top);
  if (need) ws = empty({(int64_t)need}, x, at::kByte);
  check(c.logprobs(data(x), code, size(M), size(V), ldl, static_cast<const int64_t *>(data(tokens)), (int)top,
                   static_cast<float *>(data(lp)), static_cast<float *>(data(ent)), static_cast<float *>(data(tl)),
                   static_cast<int64_t *>(data(tt)), data(ws), need, pointer(a[0])));
  return Py_BuildValue("NNNN", wrap(lp), wrap(ent), wrap(tl), wrap(tt));
}

// bind(address, ...): the C functions in the order of `c`
PyObject *bind(PyObject *const *a) {
  void **to = reinterpret_cast<void **>(&c);
  for (int i = 0; i < 7; ++i) to[i] = pointer(a[i]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    at::AutoDispatchBelowADInplaceOrView forward_only;
    return F(args);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 7>("bind"),
                         method<quantize, 3>("quantize"),
                         method<dequantize, 10>("dequantize"),
                         method<matmul, 15>("matmul"),
                         method<rmsnorm, 9>("rmsnorm"),
                         method<logprobs, 4>("logprobs"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mnb_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mnb_ops(void) { return PyModule_Create(&module); }
