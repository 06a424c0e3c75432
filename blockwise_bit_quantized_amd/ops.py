"""Binding of the operators beside MatMulNBits (``include/mnb_ops.h``): microscaled (MX)
quantisation and product, the root-mean-square norm with the residual's addition and MX
output, and log probabilities over logits.

The C calls keep their names (``mnb_mx_quantize`` ...) on plain integers; ``mx_quantize``,
``mx_dequantize``, ``mx_tensor``, ``mx_pack``, ``mx_matmul``, ``rmsnorm`` and ``logprobs``
marshal torch tensors into them; what they check and allocate is done in the native module
_mnb_ops (csrc/binding.cpp), as a single-token call is bound by the host.  Everything here is
forward only, like the rest of the package.  Scratch of a call comes from torch's allocator on
the current stream, so calls on several streams, and graph captures, need no workspace of
their own.
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

_OK = 0
lib: Any = None
_ext: Any = None
_status_text: Any = None


class _NotBuilt:
    """In the place of a native module that could not be imported: every use of it says why."""

    def __init__(self, cause):
        self._cause = cause

    def __getattr__(self, name):
        raise ImportError("the torch calls of the operators need the module _mnb_ops, built for this Python and torch: "
                          "run `python blockwise_bit_quantized_amd/build.py` (%s)" % self._cause) from self._cause


def _bind(library, status_text):
    """Called once by the package with its loaded library."""
    global lib, _ext, _status_text
    lib, _status_text = library, status_text
    P, I, L, S, F = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
    sizes = C.POINTER(S)
    for name, res, args in (
            ("mnb_mx_quantize", I, [P, I, I, I, L, I, P, L, P, L, P]),
            ("mnb_mx_dequantize", I, [P, L, P, L, I, I, I, P, I, L, P]),
            ("mnb_mx_packed_sizes", I, [I, I, sizes, sizes]),
            ("mnb_mx_pack", I, [P, L, P, L, I, I, P, P, P]),
            ("mnb_mx_matmul", I, [P, L, P, L, I, P, P, P, P, I, I, I, I, P]),
            ("mnb_mx_describe_route", I, [I, I, I, I, C.c_char_p, S]),
            ("mnb_rmsnorm", I, [P, L, P, L, P, F, I, I, I, P, L, P, L, I, P, L, P, L, P]),
            ("mnb_logprobs_workspace_bytes", S, [I, I, I, I]),
            ("mnb_logprobs", I, [P, I, I, I, L, P, I, P, P, P, P, P, S, P]),
            ("mnb_ops_version", I, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    if torch is not None:
        try:
            from . import _mnb_ops as _ext   # built with the library; there is no other path
        except ImportError as e:             # MatMulNBits and the C calls do not need it
            _ext = _NotBuilt(e)
            return
        _ext.bind(*(C.cast(getattr(lib, n), P).value for n in (
            "mnb_mx_quantize", "mnb_mx_dequantize", "mnb_mx_matmul", "mnb_rmsnorm",
            "mnb_logprobs", "mnb_logprobs_workspace_bytes", "mnb_status_string")))


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


def _run(f, t, *args):
    """f(stream, t, *args) on the current stream of t's device, with that device current."""
    try:
        i = t.get_device()
    except AttributeError:
        i = -1
    if i < 0:
        return f(0, t, *args)            # refused there, after the other checks
    # the stream's handle alone: building torch's Stream object costs as much as half a launch
    if i == torch._C._cuda_getDevice():
        return f(torch._C._cuda_getCurrentRawStream(i), t, *args)
    with torch.cuda.device(i):
        return f(torch._C._cuda_getCurrentRawStream(i), t, *args)


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
        _ld(scales, "MX scales")
        if scales.shape != (rows, K // 32) or scales.device != codes.device:
            raise ValueError("MX scales must be [%d, %d] on %s, got %s on %s"
                             % (rows, K // 32, codes.device, tuple(scales.shape), scales.device))
        need = _scale_row(K)
        # the row distance counts for one row too, as its scales are read in 16-byte pieces
        lds = scales.stride(0) if rows > 1 else need
        if K and rows and (lds % 16 or lds < need or scales.untyped_storage().nbytes() - scales.storage_offset()
                           < (rows - 1) * lds + need):
            raise ValueError("the rows of MX scales must lie a multiple of 16 bytes and at least %d apart "
                             "(mx_tensor lays them out so)" % need)
        self.codes, self.scales, self.fmt, self.rows, self.K, self.ldc, self.lds = codes, scales, fmt, rows, K, ldc, lds

    def __repr__(self):
        return "MxTensor([%d, %d], %s, %s)" % (self.rows, self.K, "FP4" if self.fmt == MNB_MX_FP4 else "FP8",
                                               self.codes.device)


def _made(codes, scales, fmt, ldc, lds, rows, K):
    """An MxTensor that a call here has just laid out."""
    q = object.__new__(MxTensor)
    q.codes, q.scales, q.fmt, q.rows, q.K, q.ldc, q.lds = codes, scales, fmt, rows, K, ldc, lds
    return q


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
    codes, scales, ldc, lds, rows, K = _run(_ext.quantize, x, fmt)
    return _made(codes, scales, fmt, ldc, lds, rows, K)


def mx_dequantize(q: MxTensor, dtype=None, out=None):
    """The values of an MX tensor in ``dtype`` (fp16 by default), each rounded once."""
    return _run(_ext.dequantize, q.codes, q.scales, q.fmt, q.rows, q.K, q.ldc, q.lds, dtype or torch.float16, out)


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
    if not q.codes.is_cuda:
        raise ValueError("tensors must be on a GPU, got %s" % q.codes.device)
    _run(lambda stream, codes: _check(lib.mnb_mx_pack(codes.data_ptr(), q.ldc, q.scales.data_ptr(), q.lds, q.rows, q.K,
                                                      w.wq.data_ptr(), w.sc.data_ptr(), stream)), q.codes)
    return w


def mx_matmul(x: MxTensor, w: MxWeight, bias=None, dtype=None, out=None):
    """Y [M, N] = x . w^T (+ bias [N]) in ``dtype`` (fp16 by default, or bf16; the bias's type too),
    rounded once; x FP8 or FP4 from mx_quantize, rmsnorm or mx_tensor.  FP4 x is summed as exactly as
    32 bits allow; with FP8 x the matrix instruction keeps fewer bits (an error of at most 2^-12 of
    the sum of |x| |w|, 2^-16 to 2^-22 in measurements)."""
    return _run(_ext.matmul, x.codes, x.scales, x.fmt, x.rows, x.K, x.ldc, x.lds, w.wq, w.sc, w.N, w.K, bias,
                dtype or torch.float16, out)


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
    y, h, codes, scales, ldc, lds, rows, K = _run(_ext.rmsnorm, x, weight, eps, residual, fmt, keep16, out, hidden)
    return Normed(y, None if fmt is None else _made(codes, scales, fmt, ldc, lds, rows, K), h)


class LogProbs(NamedTuple):
    logprob: Any        # fp32 [M] or None
    entropy: Any        # fp32 [M]
    top_logprobs: Any   # fp32 [M, top] or None
    top_tokens: Any     # int64 [M, top] or None


def logprobs(logits, tokens=None, top: int = 0) -> LogProbs:
    """For each row of logits [M, V] (fp16, bf16 or fp32): the log probability of tokens[m]
    (int64; 0 for a negative token, NaN for one past V), the entropy, and the ``top`` (at most 32)
    likeliest tokens in falling order, equal ones by the lower index."""
    return LogProbs(*_run(_ext.logprobs, logits, tokens, top))
