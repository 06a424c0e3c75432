"""Binding of the operators beside MatMulNBits (``include/mnb_ops.h``): microscaled (MX)
quantisation and product, the root-mean-square norm with the residual's addition and MX
output, and log probabilities over logits.

The C calls keep their names (``mnb_mx_quantize`` ...) on plain integers; ``mx_quantize``,
``mx_dequantize``, ``mx_tensor``, ``mx_pack``, ``mx_matmul``, ``rmsnorm`` and ``logprobs``
marshal torch tensors into them.  Everything here is forward only, like the rest of the
package.  Scratch of a call comes from torch's allocator on the current stream, so calls
on several streams, and graph captures, need no workspace of their own.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Any, NamedTuple

try:
    import torch
except ImportError:      # the C calls on plain integers need no torch, as in the package itself
    torch = None

MNB_F16, MNB_BF16, MNB_F32 = 0, 1, 2
MNB_MX_FP4, MNB_MX_FP8 = 0, 1
MNB_LOGPROBS_MAX_TOP = 32

_DTYPES = {torch.float16: MNB_F16, torch.bfloat16: MNB_BF16, torch.float32: MNB_F32} if torch else {}
_OK = 0
lib: Any = None
_status_text: Any = None


def _bind(library, status_text):
    """Called once by the package with its loaded library."""
    global lib, _status_text
    lib, _status_text = library, status_text
    P, I, L, S, F = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
    sizes = C.POINTER(S)
    for name, res, args in (
            ("mnb_mx_quantize", I, [P, I, I, I, L, I, P, L, P, L, P]),
            ("mnb_mx_dequantize", I, [P, L, P, L, I, I, I, P, I, L, P]),
            ("mnb_mx_packed_sizes", I, [I, I, sizes, sizes]),
            ("mnb_mx_pack", I, [P, L, P, L, I, I, P, P, P]),
            ("mnb_mx_workspace_bytes", S, [I, I, I, I]),
            ("mnb_mx_matmul", I, [P, L, P, L, I, P, P, P, P, I, I, I, I, P, S, P]),
            ("mnb_mx_describe_route", I, [I, I, I, I, C.c_char_p, S]),
            ("mnb_rmsnorm", I, [P, L, P, L, P, F, I, I, I, P, L, P, L, I, P, L, P, L, P]),
            ("mnb_logprobs_workspace_bytes", S, [I, I, I, I]),
            ("mnb_logprobs", I, [P, I, I, I, L, P, I, P, P, P, P, P, S, P]),
            ("mnb_ops_version", I, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ---------------------------------------------------------------------------------------
# The C ABI under its own names (integers for pointers and the stream)
# ---------------------------------------------------------------------------------------


def mnb_ops_version() -> int:
    return lib.mnb_ops_version()


def mnb_mx_quantize(*args) -> int:
    return lib.mnb_mx_quantize(*args)


def mnb_mx_dequantize(*args) -> int:
    return lib.mnb_mx_dequantize(*args)


def mnb_mx_packed_sizes(N, K):
    a, b = C.c_size_t(), C.c_size_t()
    st = lib.mnb_mx_packed_sizes(N, K, C.byref(a), C.byref(b))
    return st, a.value, b.value


def mnb_mx_pack(*args) -> int:
    return lib.mnb_mx_pack(*args)


def mnb_mx_workspace_bytes(M, N, K, fmt) -> int:
    return lib.mnb_mx_workspace_bytes(M, N, K, fmt)


def mnb_mx_matmul(*args) -> int:
    return lib.mnb_mx_matmul(*args)


def mnb_mx_describe_route(M, N, K, fmt):
    buf = C.create_string_buffer(256)
    st = lib.mnb_mx_describe_route(M, N, K, fmt, buf, 256)
    return st, buf.value.decode()


def mnb_rmsnorm(*args) -> int:
    return lib.mnb_rmsnorm(*args)


def mnb_logprobs_workspace_bytes(M, V, dtype, top) -> int:
    return lib.mnb_logprobs_workspace_bytes(M, V, dtype, top)


def mnb_logprobs(*args) -> int:
    return lib.mnb_logprobs(*args)


# ---------------------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------------------


def _check(st: int):
    if st != _OK:
        raise RuntimeError(_status_text(st))


def _call(dev, f, *args):
    """f(*args, stream) on the current stream of ``dev``, with ``dev`` current."""
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU, got %s" % dev)
    if dev.index == torch.cuda.current_device():
        st = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    if st != _OK:
        raise RuntimeError(_status_text(st))


def _rows(t, name, dtype=None, shape=None, dev=None):
    """A 2-D tensor whose rows are contiguous and do not overlap; returns its row distance."""
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dev is not None and t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    n, k = t.shape
    ld, inner = t.stride()
    if k > 1 and inner != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    if n <= 1:
        return max(k, 1)
    if ld < k:
        raise ValueError("the rows of %s must not overlap" % name)
    return ld


def _float_type(t, name, f32=True):
    code = _DTYPES.get(t.dtype)
    if code is None or (code == MNB_F32 and not f32):
        raise TypeError("%s must be float16%s, got %s" % (name, ", bfloat16 or float32" if f32 else " or bfloat16", t.dtype))
    return code


def _vector(t, name, dtype, n, dev):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous [%d], got shape %s" % (name, n, tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _blocks(K, name="the last axis"):
    if K % 32:
        raise ValueError("%s must be a multiple of 32, got %d" % (name, K))


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass
class MxTensor:
    """An MX tensor [rows, K]: ``codes`` uint8 [rows, K / 2] (MNB_MX_FP4, even k in the low
    nibble) or [rows, K] (MNB_MX_FP8; ``codes.view(torch.float8_e4m3fn)`` are its elements),
    ``scales`` uint8 [rows, K / 32] (``scales.view(torch.float8_e8m0fnu)``), whose rows lie a
    multiple of 16 bytes and at least 16 ceil(K / 512) apart."""
    codes: Any
    scales: Any
    fmt: int

    @property
    def K(self) -> int:
        return self.codes.shape[1] * (2 if self.fmt == MNB_MX_FP4 else 1)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    def check(self, dev):
        """(row distance of the codes, of the scales) after checking both tensors."""
        if self.fmt not in (MNB_MX_FP4, MNB_MX_FP8):
            raise ValueError("unknown MX format %r" % (self.fmt,))
        K = self.K
        ldc = _rows(self.codes, "MX codes", torch.uint8, None, dev)
        _blocks(K, "the last axis of an MX tensor")
        s = self.scales
        _rows(s, "MX scales", torch.uint8, (self.rows, K // 32), dev)
        if K == 0 or self.rows == 0:
            return 0, 0
        need = -(-K // 512) * 16
        # the row distance counts for one row too, as its scales are read in 16-byte pieces
        lds = s.stride(0) if self.rows > 1 else need
        if lds % 16 or lds < need or s.untyped_storage().nbytes() - s.storage_offset() < (self.rows - 1) * lds + need:
            raise ValueError("the rows of MX scales must lie a multiple of 16 bytes and at least %d apart "
                             "(mx_tensor lays them out so)" % need)
        if self.rows <= 1:
            ldc = -(-self.codes.shape[1] // 16) * 16
        return ldc, lds


def _new_scales(rows, K, dev):
    return torch.empty((rows, -(-K // 512) * 16), dtype=torch.uint8, device=dev)[:, :K // 32]


def _new_mx(rows, K, fmt, dev):
    if fmt not in (MNB_MX_FP4, MNB_MX_FP8):
        raise ValueError("unknown MX format %r" % (fmt,))
    return MxTensor(torch.empty((rows, K // 2 if fmt == MNB_MX_FP4 else K), dtype=torch.uint8, device=dev),
                    _new_scales(rows, K, dev), fmt)


def mx_tensor(codes, scales, fmt: int) -> MxTensor:
    """An MxTensor of existing codes and scales (uint8, as a checkpoint holds them); scales
    whose rows are not spaced as MxTensor needs are copied."""
    t = MxTensor(codes, scales, fmt)
    if fmt not in (MNB_MX_FP4, MNB_MX_FP8):
        raise ValueError("unknown MX format %r" % (fmt,))
    if codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("codes and scales must be 2-D")
    rows, K = t.rows, t.K
    _blocks(K, "the last axis of an MX tensor")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError("codes and scales must be uint8")
    if tuple(scales.shape) != (rows, K // 32) or scales.device != codes.device:
        raise ValueError("scales must be [%d, %d] beside the codes, got %s" % (rows, K // 32, tuple(scales.shape)))
    need = -(-K // 512) * 16
    if (K // 32 > 1 and scales.stride(1) != 1) or scales.stride(0) % 16 or scales.stride(0) < need or \
            scales.data_ptr() % 16 or \
            scales.untyped_storage().nbytes() - scales.storage_offset() < (rows - 1) * scales.stride(0) + need:
        t.scales = _new_scales(rows, K, codes.device)
        t.scales.copy_(scales)
    t.check(codes.device)
    return t


def mx_quantize(x, fmt: int = MNB_MX_FP4) -> MxTensor:
    """x [M, K] (fp16, bf16 or fp32, K a multiple of 32) to MX: one power-of-two scale for
    each 32 elements, 2^(floor(log2 max|x|) - 2 (FP4) or - 8 (FP8)), elements rounded to
    nearest even and clamped.  A block with an infinity or NaN stands for NaN throughout."""
    code = _float_type(x, "x")
    ldx = _rows(x, "x")
    M, K = x.shape
    _blocks(K, "the last axis of x")
    dev = x.device
    q = _new_mx(M, K, fmt, dev)
    _call(dev, lib.mnb_mx_quantize, x.data_ptr(), code, M, K, ldx, fmt, q.codes.data_ptr(), q.codes.shape[1],
          q.scales.data_ptr(), -(-K // 512) * 16)
    return q


def mx_dequantize(q: MxTensor, dtype=None, out=None):
    """The values of an MX tensor in ``dtype`` (fp16 by default), each rounded once."""
    dtype = dtype or torch.float16
    dev = q.codes.device
    ldc, lds = q.check(dev)
    M, K = q.rows, q.K
    y = out if out is not None else torch.empty((M, K), dtype=dtype, device=dev)
    ldy = _rows(y, "out", dtype, (M, K), dev)
    _call(dev, lib.mnb_mx_dequantize, q.codes.data_ptr(), ldc, q.scales.data_ptr(), lds, q.fmt, M, K, y.data_ptr(),
          _float_type(y, "out"), ldy)
    return y


@dataclass
class MxWeight:
    """An FP4 weight [N, K] in the layout of mx_matmul."""
    wq: Any             # torch.uint8 device tensor
    sc: Any             # torch.uint8 device tensor
    N: int
    K: int

    def check(self, dev):
        wqb, scb = _packed_sizes(self.N, self.K)
        for t, name, n in ((self.wq, "packed codes", wqb), (self.sc, "packed scales", scb)):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != dev or t.numel() < n:
                raise ValueError("%s must be a contiguous uint8 tensor of at least %d bytes on %s" % (name, n, dev))


def _packed_sizes(N, K):
    if N < 0 or K < 0 or K % 32 or K >= 1 << 25:
        _check(mnb_mx_packed_sizes(N, K)[0])
    groups = (N + 63) // 64
    return groups * ((K + 127) // 128) * 4096, groups * ((K + 511) // 512) * 1024


def mx_pack(q: MxTensor) -> MxWeight:
    """An FP4 tensor [N, K] (mx_quantize, or mx_tensor of a checkpoint's) packed for mx_matmul."""
    if q.fmt != MNB_MX_FP4:
        raise ValueError("weights are packed from MNB_MX_FP4")
    dev = q.codes.device
    ldc, lds = q.check(dev)
    N, K = q.rows, q.K
    st, wqb, scb = mnb_mx_packed_sizes(N, K)
    _check(st)
    w = MxWeight(torch.empty(wqb, dtype=torch.uint8, device=dev), torch.empty(scb, dtype=torch.uint8, device=dev), N, K)
    _call(dev, lib.mnb_mx_pack, q.codes.data_ptr(), ldc, q.scales.data_ptr(), lds, N, K, w.wq.data_ptr(), w.sc.data_ptr())
    return w


def mx_matmul(x: MxTensor, w: MxWeight, bias=None, dtype=None, out=None):
    """Y [M, N] = x . w^T (+ bias [N]) in ``dtype`` (fp16 by default, or bf16; the bias's type too),
    summed in 32 bits and rounded once; x FP8 or FP4 from mx_quantize, rmsnorm or mx_tensor."""
    dtype = dtype or torch.float16
    dev = x.codes.device
    ldc, lds = x.check(dev)
    M, K, N = x.rows, x.K, w.N
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    w.check(dev)
    if out is None:
        y = torch.empty((M, N), dtype=dtype, device=dev)
    else:
        y = out
        if y.dtype != dtype or tuple(y.shape) != (M, N) or not y.is_contiguous() or y.device != dev:
            raise ValueError("out must be a contiguous %s [%d, %d] on %s" % (dtype, M, N, dev))
    code = _float_type(y, "the output", f32=False)
    if bias is not None:
        _vector(bias, "bias", dtype, N, dev)
    need = lib.mnb_mx_workspace_bytes(M, N, K, x.fmt)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, lib.mnb_mx_matmul, x.codes.data_ptr(), ldc, x.scales.data_ptr(), lds, x.fmt, w.wq.data_ptr(),
          w.sc.data_ptr(), _ptr(bias), y.data_ptr(), code, M, N, K, _ptr(ws), need)
    return y


class Normed(NamedTuple):
    y: Any              # 16-bit output or None
    q: Any              # MxTensor or None
    hidden: Any         # x + residual, or None without a residual


def rmsnorm(x, weight, eps: float = 1e-6, residual=None, fmt: int | None = None, keep16: bool = False, out=None,
            hidden=None) -> Normed:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight for each row of x [M, K] (fp16 or
    bf16).  Without ``fmt`` y comes in x's type; with it as an MxTensor (K a multiple of 32),
    and in x's type too with ``keep16`` (an adapter's projection wants it).  ``hidden`` (given a
    residual) receives h in x's type and may be ``residual`` or ``x`` itself; ``out`` receives y
    and may be ``x``.  Each output is rounded once from 32 bits."""
    code = _float_type(x, "x", f32=False)
    ldx = _rows(x, "x")
    M, K = x.shape
    dev, dtype, shape = x.device, x.dtype, x.shape
    _vector(weight, "weight", dtype, K, dev)
    ldr = ldh = ldy = ldc = lds = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dtype, shape, dev)
        if hidden is None:
            hidden, ldh = torch.empty((M, K), dtype=dtype, device=dev), K
        else:
            ldh = _rows(hidden, "hidden", dtype, shape, dev)
    elif hidden is not None:
        raise ValueError("hidden needs a residual")
    y = q = None
    if fmt is None or keep16 or out is not None:
        if out is None:
            y, ldy = torch.empty((M, K), dtype=dtype, device=dev), K
        else:
            y, ldy = out, _rows(out, "out", dtype, shape, dev)
    if fmt is not None:
        _blocks(K, "the last axis of x")
        q = _new_mx(M, K, fmt, dev)
        ldc, lds = q.codes.shape[1], -(-K // 512) * 16
    _call(dev, lib.mnb_rmsnorm, x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), eps, code, M, K, _ptr(hidden),
          ldh, _ptr(y), ldy, fmt or 0, q.codes.data_ptr() if q else None, ldc, q.scales.data_ptr() if q else None, lds)
    return Normed(y, q, hidden)


class LogProbs(NamedTuple):
    logprob: Any        # fp32 [M] or None
    entropy: Any        # fp32 [M]
    top_logprobs: Any   # fp32 [M, top] or None
    top_tokens: Any     # int64 [M, top] or None


def logprobs(logits, tokens=None, top: int = 0) -> LogProbs:
    """For each row of logits [M, V] (fp16, bf16 or fp32): the log probability of tokens[m]
    (int64; 0 for a negative token, NaN for one past V), the entropy, and the ``top`` (at most 32)
    likeliest tokens in falling order, equal ones by the lower index."""
    code = _float_type(logits, "logits")
    ldl = _rows(logits, "logits")
    M, V = logits.shape
    dev = logits.device
    if not 0 <= top <= min(MNB_LOGPROBS_MAX_TOP, V):
        raise ValueError("top must be from 0 to %d, got %d" % (min(MNB_LOGPROBS_MAX_TOP, V), top))
    if V == 0 and M > 0:
        raise ValueError("logits have no columns")
    lp = None
    if tokens is not None:
        _vector(tokens, "tokens", torch.int64, M, dev)
        lp = torch.empty(M, dtype=torch.float32, device=dev)
    ent = torch.empty(M, dtype=torch.float32, device=dev)
    tl = torch.empty((M, top), dtype=torch.float32, device=dev) if top else None
    tt = torch.empty((M, top), dtype=torch.int64, device=dev) if top else None
    need = lib.mnb_logprobs_workspace_bytes(M, V, code, top)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, lib.mnb_logprobs, logits.data_ptr(), code, M, V, ldl, _ptr(tokens), top, _ptr(lp), ent.data_ptr(), _ptr(tl),
          _ptr(tt), _ptr(ws), need)
    return LogProbs(lp, ent, tl, tt)
