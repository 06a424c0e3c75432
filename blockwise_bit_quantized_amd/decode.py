"""Binding of the operators of a decoding step (``include/mnb_decode.h``): a paged key/value cache held in MX FP4,
appending to it with the norms of queries and keys and the rotation in the same pass, reading it back, attention
over it, and sampling.

The C calls keep their names (``mnb_kv_append`` ...) on plain integers and the two structs; ``kv_cache``,
``kv_append``, ``kv_read``, ``kv_attention`` and ``sample`` marshal torch tensors into them through the native module
_mnb_ops, on the current stream, with scratch from torch's allocator.  Forward only, like the rest of the package.

A decoding step of a layer, and the next tokens:

    q = mnb.kv_append(q, k, v, cache, pages, lengths, rope=table, q_weight=wq, k_weight=wk)
    y = mnb.kv_attention(q, cache, pages, lengths)
    ...
    tokens = mnb.sample(logits, u, temperature=0.8, top_p=0.95)
"""
from __future__ import annotations

import ctypes as C
from typing import Any

from . import ops

try:
    import torch
except ImportError:
    torch = None

lib: Any = None


class mnb_kv_cache(C.Structure):
    _fields_ = [("data", C.c_void_p), ("page_stride", C.c_int64), ("pages", C.c_int), ("kv_heads", C.c_int),
                ("head_dim", C.c_int), ("page_size", C.c_int)]


class mnb_kv_rows(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("ldp", C.c_int64), ("lengths", C.c_void_p), ("starts", C.c_void_p),
                ("batch", C.c_int), ("width", C.c_int), ("rows", C.c_int)]


def _bind(library):
    """Called once by the package with its loaded library, after ops._bind."""
    global lib
    lib = library
    P, I, L, S, F = C.c_void_p, C.c_int, C.c_int64, C.c_size_t, C.c_float
    cache, rows = C.POINTER(mnb_kv_cache), C.POINTER(mnb_kv_rows)
    for name, res, args in (
            ("mnb_kv_page_bytes", S, [I, I, I]),
            ("mnb_kv_append", I, [cache, rows, P, L, I, P, L, P, L, I, P, I, I, I, P, P, F, P, L, P]),
            ("mnb_kv_read", I, [cache, rows, P, L, P, L, I, P]),
            ("mnb_kv_attention_workspace_bytes", S, [cache, rows, I, I]),
            ("mnb_kv_attention", I, [cache, rows, P, L, I, I, F, I, P, L, P, S, P]),
            ("mnb_kv_describe_route", I, [cache, rows, I, I, C.c_char_p, S]),
            ("mnb_sample", I, [P, I, I, I, L, P, P, F, P, I, P, F, P, F, P, P]),
            ("mnb_decode_version", I, [])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    if torch is not None and not isinstance(ops._ext, ops._NotBuilt):
        ops._ext.bind_decode(*(C.cast(getattr(lib, n), P).value for n in (
            "mnb_kv_append", "mnb_kv_read", "mnb_kv_attention", "mnb_kv_attention_workspace_bytes", "mnb_sample")))


# ---------------------------------------------------------------------------------------
# The C ABI under its own names (integers for pointers and the stream)
# ---------------------------------------------------------------------------------------


def mnb_decode_version() -> int:
    return lib.mnb_decode_version()


def mnb_kv_page_bytes(kv_heads, head_dim, page_size) -> int:
    return lib.mnb_kv_page_bytes(kv_heads, head_dim, page_size)


def mnb_kv_append(*args) -> int:
    return lib.mnb_kv_append(*args)


def mnb_kv_read(*args) -> int:
    return lib.mnb_kv_read(*args)


def mnb_kv_attention_workspace_bytes(*args) -> int:
    return lib.mnb_kv_attention_workspace_bytes(*args)


def mnb_kv_attention(*args) -> int:
    return lib.mnb_kv_attention(*args)


def mnb_kv_describe_route(cache, rows, q_heads, window):
    buf = C.create_string_buffer(256)
    st = lib.mnb_kv_describe_route(cache, rows, q_heads, window, buf, 256)
    return st, buf.value.decode()


def mnb_sample(*args) -> int:
    return lib.mnb_sample(*args)


# ---------------------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------------------


class KvCache:
    """A paged key/value cache in MX FP4: ``data`` uint8 [pages, at least mnb_kv_page_bytes], whose rows lie a
    multiple of 16 bytes apart.  A page is one row, so pages are copied, swapped out and shared as rows of ``data`` are; what a
    page holds is laid out as include/mnb_decode.h says.  Checked when it is made; ``data`` may be
    written to, but not resized."""
    __slots__ = ("data", "kv_heads", "head_dim", "page_size")

    def __init__(self, data, kv_heads: int, head_dim: int, page_size: int):
        if kv_heads < 1:
            raise ValueError("a cache needs at least one key/value head, got %d" % kv_heads)
        need = mnb_kv_page_bytes(kv_heads, head_dim, page_size)
        if need == 0:
            raise ValueError("head_dim must be 64, 96, 128, 192 or 256 and page_size a power of two from 16 to 65536, "
                             "got %d and %d" % (head_dim, page_size))
        if data.dtype != torch.uint8:
            raise TypeError("the cache's data must be uint8")
        ld = ops._ld(data, "the cache's data")
        if data.shape[1] < need or ld % 16 or data.data_ptr() % 16:
            raise ValueError("the cache's data must be [pages, at least %d] with rows a multiple of 16 bytes apart" % need)
        self.data, self.kv_heads, self.head_dim, self.page_size = data, kv_heads, head_dim, page_size

    @property
    def pages(self) -> int:
        return self.data.shape[0]

    def _args(self):
        return self.data, self.kv_heads, self.head_dim, self.page_size

    def __repr__(self):
        return "KvCache(%d pages of %d, %d heads of %d, %s)" % (self.pages, self.page_size, self.kv_heads, self.head_dim,
                                                                self.data.device)


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device=None) -> KvCache:
    """A new cache of ``pages`` pages of ``page_size`` tokens (head_dim + head_dim / 16 bytes a token and head).  Its bytes
    are not cleared: nothing reads a place that no row was appended to."""
    need = mnb_kv_page_bytes(kv_heads, head_dim, page_size)
    return KvCache(torch.empty((pages, max(need, 16)), dtype=torch.uint8, device=device or "cuda"), kv_heads, head_dim, page_size)


def rope_table(positions: int, rot: int, base: float = 10000.0, device=None, inv_freq=None):
    """The rotation table of ``kv_append``: fp32 [positions, rot], rot / 2 cosines and as many sines of position *
    base^(-2 i / rot), or of position * inv_freq[i] where frequencies are given.  The angles are taken in 64
    bits: 32 lose them at far positions."""
    if rot % 16:
        raise ValueError("rot must be a multiple of 16, got %d" % rot)
    if inv_freq is None:
        inv_freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    inv_freq = inv_freq.detach().to("cpu", torch.float64)
    if inv_freq.shape != (rot // 2,):
        raise ValueError("inv_freq must be [%d], got %s" % (rot // 2, tuple(inv_freq.shape)))
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv_freq
    return torch.cat((angle.cos(), angle.sin()), 1).float().to(device or "cuda")


def kv_append(q, k, v, cache: KvCache, pages, lengths, starts=None, rope=None, q_weight=None, k_weight=None,
              eps: float = 1e-6, interleaved: bool = False, out=None):
    """Append the rows k and v [rows, kv_heads, head_dim] (fp16 or bf16; slices of one projection's output will do) to the
    cache and return the queries, q [rows, q_heads, head_dim] (or None) taken the same way:
    over each head h = x / sqrt(mean(x^2) + eps) * weight for queries and keys where a weight [head_dim] is given, then the
    rotation of the first ``rope.shape[1]`` elements by the table's row at the row's position, in pairs (i, i + half), or
    (2 i, 2 i + 1) with ``interleaved``.  Keys, in 64 bits, and values go to MX FP4.  ``out`` receives the queries and may be q.

    Sequence b has ``lengths[b]`` tokens in the cache after the call (int32), the rows starts[b] .. starts[b + 1] - 1 last
    (``starts`` int32 [batch + 1]; None: one row each); position p lies in page ``pages[b, p // page_size]`` (int32
    [batch, width]).  A row at a negative position gives zeros and is not stored; one past the pages' width or in a page
    out of range gives NaN and is not stored; one past the table gives NaN and is stored as NaN; rows behind the last sequence are not
    written.  Positions of a call must not share a place in a page."""
    return ops._run(ops._ext.kv_append, k, q, v, *cache._args(), pages, lengths, starts, rope, q_weight, k_weight, eps,
                    interleaved, out)


def kv_read(cache: KvCache, pages, lengths, rows: int | None = None, starts=None, dtype=None, out=(None, None)):
    """(k, v) [rows, kv_heads, head_dim] in ``dtype`` (fp16 by default): the cache's values at the positions of the
    rows that ``kv_append`` takes with the same lengths and starts.  ``rows`` is their number (len(lengths) without starts);
    starts that sum the lengths read whole sequences.  Rows without a position are zeros, those out of reach
    NaN, and those behind the last sequence are not written."""
    if rows is None:
        if starts is not None:
            raise ValueError("rows is needed with starts")
        rows = len(lengths)
    return ops._run(ops._ext.kv_read, *cache._args(), pages, lengths, starts, rows, dtype or torch.float16, *out)


def kv_attention(q, cache: KvCache, pages, lengths, starts=None, scale: float | None = None, window: int = 0, out=None):
    """softmax(scale q . k) v [rows, q_heads, head_dim] in q's type (fp16 or bf16) for each row over the tokens of its
    sequence up to its own, the last ``window`` of them where window > 0; the rows are those of ``kv_append``, whose own
    tokens have been appended.  q_heads is a multiple of the cache's heads, query head h reads head h // (q_heads //
    kv_heads); scale is 1 / sqrt(head_dim) by default.  A row that sees nothing is zeros.  ``out`` may be q."""
    return ops._run(ops._ext.kv_attention, q, *cache._args(), pages, lengths, starts, scale, window, out)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None):
    """One token (int64 [M]) for each row of logits [M, V] (fp16, bf16 or fp32) from u [M] in [0, 1) (fp32).  Of
    softmax(logits / temperature) the top_k largest stay (0: all; equal ones by the lower index), of these, renormalised, the
    shortest run of largest ones that reaches top_p, of these those with at least min_p times the largest; the token is the
    first by index at which the running sum of what stays passes u times the whole.  Temperature 0 takes the largest.
    Each parameter is a number or a tensor [M] (fp32; top_k int32).  -1 where there is no distribution (a NaN,
    +infinity, or only -infinity; a NaN or negative temperature and the like)."""
    return ops._run(ops._ext.sample, logits, u, temperature, top_k, top_p, min_p, out)
