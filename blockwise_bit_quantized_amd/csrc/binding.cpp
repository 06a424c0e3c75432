// binding.cpp -- the host side of the torch binding of include/mnb_ops.h and include/mnb_decode.h (module
// _mnb_ops): checks of arguments, output and scratch allocation, and the C call, in one native call.
//
// A single-token call is bound by the host: a launch takes about 3.2 us, and the same
// steps in Python (attribute reads, allocations, ctypes) took 4 to 10 us on top of it where
// these take 2 to 3.  The module holds no state but the addresses of the C functions, which
// `bind` and `bind_decode` receive once; every function takes the stream handle first.  Forward only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <string>

#include "mnb_decode.h"

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
struct {
  decltype(&mnb_kv_append) append;
  decltype(&mnb_kv_read) read;
  decltype(&mnb_kv_attention) attention;
  decltype(&mnb_kv_attention_workspace_bytes) attention_ws;
  decltype(&mnb_sample) sample;
} d;

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

// ---- include/mnb_decode.h -----------------------------------------------------------------------

// cache: a[0..3] data, kv_heads, head_dim, page_size (its data checked where the cache was made)
struct Cache {
  at::Tensor data;
  mnb_kv_cache c{};
  explicit Cache(PyObject *const *a) : data(tensor(a[0], "the cache's data")) {
    if (data.scalar_type() != at::kByte) fail(PyExc_TypeError, "the cache's data must be uint8");
    const int64_t stride = row_distance(data, "the cache's data");
    c.data = data.data_ptr();
    c.pages = size(data.size(0));
    c.kv_heads = size(integer(a[1]));
    c.head_dim = size(integer(a[2]));
    c.page_size = size(integer(a[3]));
    c.page_stride = stride;
  }
};
// rows: a[0..2] pages, lengths, starts or None
struct Rows {
  at::Tensor pages, lengths, starts;
  mnb_kv_rows r{};
  Rows(PyObject *const *a, int64_t rows, at::Device dev)
      : pages(tensor(a[0], "pages")), lengths(tensor(a[1], "lengths")), starts(maybe_tensor(a[2], "starts")) {
    if (pages.scalar_type() != at::kInt) fail(PyExc_TypeError, "pages must be int32, got %s", at::toString(pages.scalar_type()));
    r.ldp = row_distance(pages, "pages");
    if (pages.device() != dev)
      fail(PyExc_ValueError, "pages is on %s, expected %s", pages.device().str().c_str(), dev.str().c_str());
    const int64_t batch = pages.size(0);
    vector(lengths, "lengths", at::kInt, batch, dev);
    if (starts.defined()) vector(starts, "starts", at::kInt, batch + 1, dev);
    else if (rows != batch)
      fail(PyExc_ValueError, "without starts every sequence has one row: %lld rows, %lld sequences", (long long)rows, (long long)batch);
    r.pages = static_cast<const int32_t *>(data(pages));
    r.lengths = static_cast<const int32_t *>(data(lengths));
    r.starts = static_cast<const int32_t *>(data(starts));
    r.batch = size(batch);
    r.width = size(pages.size(1));
    r.rows = size(rows);
  }
};

// The row distance of [rows, heads, head_dim] whose heads lie side by side.
int64_t heads_distance(const at::Tensor &t, const char *name, int64_t rows, int64_t heads, int64_t D) {
  if (t.dim() != 3 || (rows >= 0 && t.size(0) != rows) || (heads >= 0 && t.size(1) != heads) || t.size(2) != D)
    fail(PyExc_ValueError, "%s has shape %s, expected [%s, %s, %lld]", name, shape_of(t).c_str(), rows < 0 ? "rows" : std::to_string(rows).c_str(),
         heads < 0 ? "heads" : std::to_string(heads).c_str(), (long long)D);
  const int64_t n = t.size(0), h = t.size(1);
  if (t.stride(2) != 1 || (h > 1 && t.stride(1) != D)) fail(PyExc_ValueError, "the heads of %s must lie side by side", name);
  if (n <= 1) return h * D ? h * D : 1;
  if (t.stride(0) < h * D) fail(PyExc_ValueError, "the rows of %s must not overlap", name);
  return t.stride(0);
}
int64_t heads_beside(const at::Tensor &t, const char *name, at::ScalarType type, int64_t rows, int64_t heads, int64_t D, at::Device dev) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s must be %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
  if (t.device() != dev)
    fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
  return heads_distance(t, name, rows, heads, D);
}

// kv_append(stream, k, q or None, v, cache x 4, pages, lengths, starts, table, q_weight, k_weight, eps, interleaved, out) -> q
PyObject *kv_append(PyObject *const *a) {
  const at::Tensor k = tensor(a[1], "k"), q = maybe_tensor(a[2], "q"), v = tensor(a[3], "v"), table = maybe_tensor(a[11], "rope"),
                   qw = maybe_tensor(a[12], "q_weight"), kw = maybe_tensor(a[13], "k_weight");
  at::Tensor y = maybe_tensor(a[16], "out");
  const Cache cache(a + 4);
  const int D = cache.c.head_dim;
  const int code = float_type(k, "k", false);
  const at::ScalarType type = k.scalar_type();
  const at::Device dev = k.device();
  const int64_t ldk = heads_distance(k, "k", -1, cache.c.kv_heads, D), rows = k.size(0);
  const int64_t ldv = heads_beside(v, "v", type, rows, cache.c.kv_heads, D, dev);
  int64_t ldq = 0, ldo = 0, heads = 0;
  if (q.defined()) {
    ldq = heads_beside(q, "q", type, rows, -1, D, dev);
    heads = q.size(1);
    if (y.defined()) ldo = heads_beside(y, "out", type, rows, heads, D, dev);
    else {
      y = empty({rows, heads, D}, q, type);
      ldo = heads * D;
    }
  } else if (y.defined()) {
    fail(PyExc_ValueError, "out needs q");
  }
  if (cache.data.device() != dev)
    fail(PyExc_ValueError, "the cache is on %s, expected %s", cache.data.device().str().c_str(), dev.str().c_str());
  const Rows r(a + 8, rows, dev);
  int64_t rot = 0, table_rows = 0;
  if (table.defined()) {
    if (table.scalar_type() != at::kFloat) fail(PyExc_TypeError, "rope must be float32, got %s", at::toString(table.scalar_type()));
    if (table.dim() != 2 || !table.is_contiguous() || table.device() != dev)
      fail(PyExc_ValueError, "rope must be a contiguous [positions, rotated elements] on %s", dev.str().c_str());
    table_rows = table.size(0);
    rot = table.size(1);
    if (rot % 16 || rot > D) fail(PyExc_ValueError, "rope must have a multiple of 16 and at most %d columns, got %lld", D, (long long)rot);
  }
  if (qw.defined()) vector(qw, "q_weight", type, D, dev);
  if (kw.defined()) vector(kw, "k_weight", type, D, dev);
  const double eps = PyFloat_AsDouble(a[14]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  const bool interleaved = truth(a[15]);
  on_gpu(k);
  check(d.append(&cache.c, &r.r, data(q), ldq, size(heads), data(k), ldk, data(v), ldv, code, static_cast<const float *>(data(table)),
                 size(table_rows), size(rot), interleaved, data(qw), data(kw), (float)eps, data(y), ldo, pointer(a[0])));
  written(cache.data);
  if (a[16] != Py_None) written(y);
  return wrap(y);
}

// kv_read(stream, data, kv_heads, head_dim, page_size, pages, lengths, starts, rows, dtype, k or None, v or None) -> (k, v)
PyObject *kv_read(PyObject *const *a) {
  const Cache cache(a + 1);
  const at::Device dev = cache.data.device();
  const int64_t rows = integer(a[8]), heads = cache.c.kv_heads, D = cache.c.head_dim;
  if (rows < 0) fail(PyExc_ValueError, "rows must not be negative, got %lld", (long long)rows);
  if (!THPDtype_Check(a[9])) fail(PyExc_TypeError, "dtype must be a torch dtype");
  const at::ScalarType type = reinterpret_cast<THPDtype *>(a[9])->scalar_type;
  if (type_code(type) < 0) fail(PyExc_TypeError, "the output must be float16, bfloat16 or float32");
  const Rows r(a + 5, rows, dev);
  at::Tensor out[2] = {maybe_tensor(a[10], "out"), maybe_tensor(a[11], "out")};
  int64_t ld[2];
  for (int i = 0; i < 2; ++i) {
    if (out[i].defined()) ld[i] = heads_beside(out[i], "out", type, rows, heads, D, dev);
    else {
      out[i] = empty({rows, heads, D}, cache.data, type);
      ld[i] = heads * D ? heads * D : 1;
    }
  }
  on_gpu(cache.data);
  check(d.read(&cache.c, &r.r, data(out[0]), ld[0], data(out[1]), ld[1], type_code(type), pointer(a[0])));
  for (int i = 0; i < 2; ++i)
    if (a[10 + i] != Py_None) written(out[i]);
  return Py_BuildValue("NN", wrap(out[0]), wrap(out[1]));
}

// kv_attention(stream, q, cache x 4, pages, lengths, starts, scale or None, window, out) -> y
PyObject *kv_attention(PyObject *const *a) {
  const at::Tensor q = tensor(a[1], "q");
  at::Tensor y = maybe_tensor(a[11], "out"), ws;
  const Cache cache(a + 2);
  const int D = cache.c.head_dim;
  const int code = float_type(q, "q", false);
  const at::Device dev = q.device();
  const int64_t ldq = heads_distance(q, "q", -1, -1, D), rows = q.size(0), heads = q.size(1);
  if (cache.data.device() != dev)
    fail(PyExc_ValueError, "the cache is on %s, expected %s", cache.data.device().str().c_str(), dev.str().c_str());
  if (cache.c.kv_heads == 0 || heads % cache.c.kv_heads)
    fail(PyExc_ValueError, "%lld query heads are no multiple of %d key/value heads", (long long)heads, cache.c.kv_heads);
  const Rows r(a + 6, rows, dev);
  double scale = 1.0 / std::sqrt((double)D);
  if (a[9] != Py_None) {
    scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
  }
  const int64_t window = integer(a[10]);
  if (window < 0) fail(PyExc_ValueError, "window must not be negative, got %lld", (long long)window);
  int64_t ldy = heads * D;
  if (y.defined()) ldy = heads_beside(y, "out", q.scalar_type(), rows, heads, D, dev);
  else y = empty({rows, heads, D}, q, q.scalar_type());
  on_gpu(q);
  const int w = window > INT32_MAX ? INT32_MAX : (int)window;
  const size_t need = d.attention_ws(&cache.c, &r.r, size(heads), w);
  if (need) ws = empty({(int64_t)need}, q, at::kByte);
  check(d.attention(&cache.c, &r.r, data(q), ldq, size(heads), code, (float)scale, w, data(y), ldy, data(ws), need, pointer(a[0])));
  if (a[11] != Py_None) written(y);
  return wrap(y);
}

// a parameter of sampling: a tensor [M], or a number for all rows
struct Parameter {
  at::Tensor t;
  double number = 0;
  Parameter(PyObject *o, const char *name, at::ScalarType type, int64_t M, at::Device dev) {
    if (THPVariable_Check(o)) {
      t = THPVariable_Unpack(o);
      vector(t, name, type, M, dev);
      return;
    }
    if (type == at::kInt) {
      const int64_t v = integer(o);
      number = (double)(v > INT32_MAX ? INT32_MAX : v < 0 ? 0 : v);
    } else {
      number = PyFloat_AsDouble(o);
      if (number == -1.0 && PyErr_Occurred()) throw Raised();
    }
  }
};

// sample(stream, logits, u, temperature, top_k, top_p, min_p, out) -> tokens
PyObject *sample(PyObject *const *a) {
  const at::Tensor x = tensor(a[1], "logits"), u = tensor(a[2], "u");
  at::Tensor y = maybe_tensor(a[7], "out");
  const int code = float_type(x, "logits", true);
  const int64_t ldl = row_distance(x, "logits"), M = x.size(0), V = x.size(1);
  const at::Device dev = x.device();
  vector(u, "u", at::kFloat, M, dev);
  const Parameter temperature(a[3], "temperature", at::kFloat, M, dev), top_k(a[4], "top_k", at::kInt, M, dev),
      top_p(a[5], "top_p", at::kFloat, M, dev), min_p(a[6], "min_p", at::kFloat, M, dev);
  if (V == 0 && M > 0) fail(PyExc_ValueError, "logits have no columns");
  if (y.defined()) vector(y, "out", at::kLong, M, dev);
  else y = empty({M}, x, at::kLong);
  on_gpu(x);
  check(d.sample(data(x), code, size(M), size(V), ldl, static_cast<const float *>(data(u)), static_cast<const float *>(data(temperature.t)),
                 (float)temperature.number, static_cast<const int32_t *>(data(top_k.t)), (int)top_k.number,
                 static_cast<const float *>(data(top_p.t)), (float)top_p.number, static_cast<const float *>(data(min_p.t)),
                 (float)min_p.number, static_cast<int64_t *>(data(y)), pointer(a[0])));
  if (a[7] != Py_None) written(y);
  return wrap(y);
}

// bind(address, ...): the C functions in the order of `c`
PyObject *bind(PyObject *const *a) {
  void **to = reinterpret_cast<void **>(&c);
  for (int i = 0; i < 7; ++i) to[i] = pointer(a[i]);
  Py_RETURN_NONE;
}

// bind_decode(address, ...): in the order of `d`
PyObject *bind_decode(PyObject *const *a) {
  void **to = reinterpret_cast<void **>(&d);
  for (int i = 0; i < 5; ++i) to[i] = pointer(a[i]);
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
                         method<bind_decode, 5>("bind_decode"),
                         method<kv_append, 17>("kv_append"),
                         method<kv_read, 12>("kv_read"),
                         method<kv_attention, 12>("kv_attention"),
                         method<sample, 8>("sample"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mnb_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mnb_ops(void) { return PyModule_Create(&module); }
