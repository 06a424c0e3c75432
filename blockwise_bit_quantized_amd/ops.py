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
    i = dev.index
    if i is None or dev.type != "cuda":
        raise ValueError("tensors must be on a GPU, got %s" % dev)
    if i == torch.cuda.current_device():
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(i))
    if st != _OK:
        raise RuntimeError(_status_text(st))


def _raw_stream(index):
    # the handle alone: building torch's Stream object costs as much as half a launch
    return torch._C._cuda_getCurrentRawStream(index)


def _ld(t, name):
    """The row distance of a 2-D tensor whose rows are contiguous and do not overlap."""
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    n, k = t.shape
    ld, inner = t.stride()
    if inner != 1 and k > 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    if n <= 1:
        return k or 1
    if ld < k:
        raise ValueError("the rows of %s must not overlap" % name)
    return ld


def _beside(t, name, dtype, shape, dev):
    """_ld of a tensor that has to match another's type, shape and device."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    return _ld(t, name)


def _float_type(t, name, f32=True):
    code = _DTYPES.get(t.dtype)
    if code is None or (code == MNB_F32 and not f32):
        raise TypeError("%s must be float16%s, got %s" % (name, ", bfloat16 or float32" if f32 else " or bfloat16", t.dtype))
    return code


def _vector(t, name, dtype, n, dev):
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous [%d], got shape %s" % (name, n, tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _blocks(K, name):
    if K % 32:
        raise ValueError("%s must be a multiple of 32, got %d" % (name, K))


def _format(fmt):
    if fmt != MNB_MX_FP4 and fmt != MNB_MX_FP8:
        raise ValueError("unknown MX format %r" % (fmt,))


def _scale_row(K):
    return (K + 511) // 512 * 16


class MxTensor:
    """An MX tensor [rows, K]: ``codes`` uint8 [rows, K / 2] (MNB_MX_FP4, even k in the low
    nibble) or [rows, K] (MNB_MX_FP8; ``codes.view(torch.float8_e4m3fn)`` are its elements),
    ``scales`` uint8 [rows, K / 32] (``scales.view(torch.float8_e8m0fnu)``), whose rows lie a
    multiple of 16 bytes and at least 16 ceil(K / 512) apart.  Checked when it is made; the
    tensors may be written to, but not resized."""
    __slots__ = ("codes", "scales", "fmt", "rows", "K", "ldc", "lds")

    def __init__(self, codes, scales, fmt: int):
        _format(fmt)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("MX codes and scales must be uint8")
        ldc = _ld(codes, "MX codes")
        rows, per_row = codes.shape
        K = per_row * 2 if fmt == MNB_MX_FP4 else per_row
        _blocks(K, "the last axis of an MX tensor")
        _beside(scales, "MX scales", torch.uint8, (rows, K // 32), codes.device)
        need = _scale_row(K)
        # the row distance counts for one row too, as its scales are read in 16-byte pieces
        lds = scales.stride(0) if rows > 1 else need
        if K and rows and (lds % 16 or lds < need or scales.untyped_storage().nbytes() - scales.storage_offset()
                           < (rows - 1) * lds + need):
            raise ValueError("the rows of MX scales must lie a multiple of 16 bytes and at least %d apart "
                             "(mx_tensor lays them out so)" % need)
        self.codes, self.scales, self.fmt, self.rows, self.K, self.ldc, self.lds = codes, scales, fmt, rows, K, ldc, lds

    @classmethod
    def _new(cls, like, rows, K, fmt):
        """Uninitialised, on the device of ``like``."""
        _format(fmt)
        q = object.__new__(cls)
        ldc, lds = K // 2 if fmt == MNB_MX_FP4 else K, _scale_row(K)
        s = like.new_empty((rows, lds), dtype=torch.uint8)
        q.codes = like.new_empty((rows, ldc), dtype=torch.uint8)
        q.scales = s if lds == K // 32 else s[:, :K // 32]
        q.fmt, q.rows, q.K, q.ldc, q.lds = fmt, rows, K, ldc, lds
        return q

    def __repr__(self):
        return "MxTensor([%d, %d], %s, %s)" % (self.rows, self.K, "FP4" if self.fmt == MNB_MX_FP4 else "FP8",
                                               self.codes.device)


def mx_tensor(codes, scales, fmt: int) -> MxTensor:
    """An MxTensor of existing codes and scales (uint8, as a checkpoint holds them); scales
    whose rows are not spaced as MxTensor needs are copied."""
    _format(fmt)
    if codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("MX codes and scales must be 2-D")
    rows, K = codes.shape[0], codes.shape[1] * (2 if fmt == MNB_MX_FP4 else 1)
    if scales.dtype == torch.uint8 and scales.shape == (rows, K // 32):
        need, ld = _scale_row(K), scales.stride(0)
        if (K > 32 and scales.stride(1) != 1) or ld % 16 or ld < need or scales.data_ptr() % 16 or \
                scales.untyped_storage().nbytes() - scales.storage_offset() < (rows - 1) * ld + need:
            spaced = scales.new_empty((rows, need))[:, :K // 32]
            spaced.copy_(scales)
            scales = spaced
    return MxTensor(codes, scales, fmt)


def mx_quantize(x, fmt: int = MNB_MX_FP4) -> MxTensor:
    """x [M, K] (fp16, bf16 or fp32, K a multiple of 32) to MX: one power-of-two scale for
    each 32 elements, 2^(floor(log2 max|x|) - 2 (FP4) or - 8 (FP8)), elements rounded to
    nearest even and clamped.  A block with an infinity or NaN stands for NaN throughout."""
    code = _float_type(x, "x")
    ldx = _ld(x, "x")
    M, K = x.shape
    _blocks(K, "the last axis of x")
    q = MxTensor._new(x, M, K, fmt)
    _call(x.device, lib.mnb_mx_quantize, x.data_ptr(), code, M, K, ldx, fmt, q.codes.data_ptr(), q.ldc,
          q.scales.data_ptr(), q.lds)
    return q


def mx_dequantize(q: MxTensor, dtype=None, out=None):
    """The values of an MX tensor in ``dtype`` (fp16 by default), each rounded once."""
    dtype = dtype or torch.float16
    M, K = q.rows, q.K
    if out is None:
        out, ldy = q.codes.new_empty((M, K), dtype=dtype), K
    else:
        ldy = _beside(out, "out", dtype, (M, K), q.codes.device)
    _call(q.codes.device, lib.mnb_mx_dequantize, q.codes.data_ptr(), q.ldc, q.scales.data_ptr(), q.lds, q.fmt, M, K,
          out.data_ptr(), _float_type(out, "out"), ldy)
    return out


class MxWeight:
    """An FP4 weight [N, K] in the layout of mx_matmul: ``wq`` and ``sc`` uint8 device buffers of
    mnb_mx_packed_sizes bytes.  Checked when it is made."""
    __slots__ = ("wq", "sc", "N", "K")

    def __init__(self, wq, sc, N: int, K: int):
        st, wqb, scb = mnb_mx_packed_sizes(N, K)
        _check(st)
        for t, name, n in ((wq, "packed codes", wqb), (sc, "packed scales", scb)):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != wq.device or t.numel() < n:
                raise ValueError("%s must be a contiguous uint8 tensor of at least %d bytes on %s" % (name, n, wq.device))
        self.wq, self.sc, self.N, self.K = wq, sc, N, K


def mx_pack(q: MxTensor) -> MxWeight:
    """An FP4 tensor [N, K] (mx_quantize, or mx_tensor of a checkpoint's) packed for mx_matmul."""
    if q.fmt != MNB_MX_FP4:
        raise ValueError("weights are packed from MNB_MX_FP4")
    st, wqb, scb = mnb_mx_packed_sizes(q.rows, q.K)
    _check(st)
    w = MxWeight(q.codes.new_empty(wqb), q.codes.new_empty(scb), q.rows, q.K)
    _call(q.codes.device, lib.mnb_mx_pack, q.codes.data_ptr(), q.ldc, q.scales.data_ptr(), q.lds, q.rows, q.K,
          w.wq.data_ptr(), w.sc.data_ptr())
    return w


def mx_matmul(x: MxTensor, w: MxWeight, bias=None, dtype=None, out=None):
    """Y [M, N] = x . w^T (+ bias [N]) in ``dtype`` (fp16 by default, or bf16; the bias's type too),
    summed in 32 bits and rounded once; x FP8 or FP4 from mx_quantize, rmsnorm or mx_tensor."""
    codes = x.codes
    dev, M, K, N = codes.device, x.rows, x.K, w.N
    dtype = dtype or torch.float16
    code = _DTYPES.get(dtype)
    if code is None or code == MNB_F32:
        raise TypeError("the output must be float16 or bfloat16, got %s" % dtype)
    if K != w.K:
        raise ValueError("x has K=%d, weight has K=%d" % (K, w.K))
    if w.wq.device != dev:
        raise ValueError("the weight is on %s, expected %s" % (w.wq.device, dev))
    if out is None:
        out = codes.new_empty((M, N), dtype=dtype)
    elif out.dtype != dtype or out.shape != (M, N) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous %s [%d, %d] on %s" % (dtype, M, N, dev))
    if bias is not None:
        _vector(bias, "bias", dtype, N, dev)
        bias = bias.data_ptr()
    need = lib.mnb_mx_workspace_bytes(M, N, K, x.fmt)
    ws = codes.new_empty(need) if need else None
    _call(dev, lib.mnb_mx_matmul, codes.data_ptr(), x.ldc, x.scales.data_ptr(), x.lds, x.fmt, w.wq.data_ptr(),
          w.sc.data_ptr(), bias, out.data_ptr(), code, M, N, K, ws.data_ptr() if need else None, need)
    return out


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
    ldx = _ld(x, "x")
    shape, dev, dtype = x.shape, x.device, x.dtype
    M, K = shape
    _vector(weight, "weight", dtype, K, dev)
    rp = hp = yp = cp = sp = y = q = None
    ldr = ldh = ldy = ldc = lds = 0
    if residual is not None:
        ldr = _beside(residual, "residual", dtype, shape, dev)
        if hidden is None:
            hidden, ldh = x.new_empty(shape), K
        else:
            ldh = _beside(hidden, "hidden", dtype, shape, dev)
        rp, hp = residual.data_ptr(), hidden.data_ptr()
    elif hidden is not None:
        raise ValueError("hidden needs a residual")
    if fmt is None or keep16 or out is not None:
        if out is None:
            y, ldy = x.new_empty(shape), K
        else:
            y, ldy = out, _beside(out, "out", dtype, shape, dev)
        yp = y.data_ptr()
    if fmt is not None:
        _blocks(K, "the last axis of x")
        q = MxTensor._new(x, M, K, fmt)
        cp, ldc, sp, lds = q.codes.data_ptr(), q.ldc, q.scales.data_ptr(), q.lds
    _call(dev, lib.mnb_rmsnorm, x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), eps, code, M, K, hp, ldh, yp, ldy,
          fmt or 0, cp, ldc, sp, lds)
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
    ldl = _ld(logits, "logits")
    M, V = logits.shape
    dev = logits.device
    if not 0 <= top <= min(MNB_LOGPROBS_MAX_TOP, V):
        raise ValueError("top must be from 0 to %d, got %d" % (min(MNB_LOGPROBS_MAX_TOP, V), top))
    if V == 0 and M > 0:
        raise ValueError("logits have no columns")
    tp = lp = lpp = tl = tlp = tt = ttp = ws = None
    if tokens is not None:
        _vector(tokens, "tokens", torch.int64, M, dev)
        lp = logits.new_empty(M, dtype=torch.float32)
        tp, lpp = tokens.data_ptr(), lp.data_ptr()
    ent = logits.new_empty(M, dtype=torch.float32)
    if top:
        tl, tt = logits.new_empty((M, top), dtype=torch.float32), logits.new_empty((M, top), dtype=torch.int64)
        tlp, ttp = tl.data_ptr(), tt.data_ptr()
    need = lib.mnb_logprobs_workspace_bytes(M, V, code, top)
    if need:
        ws = logits.new_empty(need, dtype=torch.uint8)
    _call(dev, lib.mnb_logprobs, logits.data_ptr(), code, M, V, ldl, tp, top, lpp, ent.data_ptr(), tlp, ttp,
          ws.data_ptr() if need else None, need)
    return LogProbs(lp, ent, tl, tt)
