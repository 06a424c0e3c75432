"""Host-side checks of include/mnb_ops.h that need no GPU: exported names, sizes, routes,
argument validation before any device call, the torch binding's refusals, and the
references that the GPU tests compare with (pinned to torch's own casts and to exact
arithmetic)."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

import _ops_ref as ref
from _util import ROOT, ensure_lib

mnb = ensure_lib()
torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, ALIAS = 0, 1, 2, 3, 4, 5
P = [(i + 1) << 40 for i in range(12)]     # far apart, never dereferenced


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mnb_ops.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mnb_[a-z_]+)\s*\(", text)))
    assert len(names) == 10
    for n in names:
        assert hasattr(mnb.lib, n) and callable(getattr(mnb, n)), n
    assert mnb.mnb_ops_version() == 100


def test_packed_sizes_and_routes():
    for N, K in ((1, 32), (64, 128), (65, 160), (1000, 1056), (49152, 576)):
        st, wq, sc = mnb.mnb_mx_packed_sizes(N, K)
        assert (st, wq, sc) == (OK, -(-N // 64) * -(-K // 128) * 4096, -(-N // 64) * -(-K // 512) * 1024)
    assert mnb.mnb_mx_packed_sizes(64, 40)[0] == UNSUPPORTED
    assert mnb.mnb_mx_packed_sizes(-1, 64)[0] == INVALID
    assert mnb.mnb_mx_packed_sizes(64, 1 << 25)[0] == UNSUPPORTED

    def route(*a):
        st, text = mnb.mnb_mx_describe_route(*a)
        assert st == OK
        return text
    assert route(0, 64, 64, 0) == "noop" and route(4, 64, 0, 1) == "fill"
    assert route(1, 8192, 2048, 1).startswith("mx_gemv_fp8") and route(32, 8192, 2048, 0).startswith("mx_gemv_fp4")
    assert route(33, 8192, 2048, 0) == "mx_gemm_fp4 tile=64x128"
    assert route(1024, 4096, 4096, 0).endswith("tile=128x128") and route(8192, 9728, 2560, 1).endswith("tile=128x256")
    assert mnb.mnb_mx_describe_route(1, 64, 64, 2)[0] == INVALID


def quant(X=P[0], dt=0, M=4, K=64, ldx=64, fmt=1, c=P[1], ldc=64, s=P[2], lds=16):
    return mnb.mnb_mx_quantize(X, dt, M, K, ldx, fmt, c, ldc, s, lds, None)


def test_quantize_validation():
    assert quant(M=0, X=None) == OK and quant(K=0, X=None) == OK
    assert quant(M=-1) == INVALID and quant(dt=3) == INVALID and quant(fmt=2) == INVALID
    assert quant(K=48) == UNSUPPORTED
    assert quant(X=None) == INVALID and quant(c=None) == INVALID and quant(s=None) == INVALID
    assert quant(ldx=32) == INVALID and quant(ldc=32) == INVALID and quant(lds=0) == INVALID
    assert quant(K=576, ldx=576, ldc=576, lds=16) == INVALID          # 576 / 512: two pieces of 16
    assert quant(X=P[0] + 2) == MISALIGNED and quant(c=P[1] + 8) == MISALIGNED and quant(s=P[2] + 4) == MISALIGNED
    assert quant(ldx=68) == MISALIGNED and quant(ldc=72) == MISALIGNED and quant(lds=24) == MISALIGNED
    assert quant(c=P[0]) == ALIAS and quant(s=P[0] + 64) == ALIAS and quant(s=P[1] + 16) == ALIAS
    f = mnb.mnb_mx_dequantize
    assert f(P[0], 64, P[1], 16, 1, 4, 64, None, 0, 64, None) == INVALID
    assert f(P[0], 64, P[1], 16, 1, 4, 64, P[0], 0, 64, None) == ALIAS
    assert f(P[0], 64, P[1], 16, 1, 4, 64, P[2], 0, 66, None) == MISALIGNED
    g = mnb.mnb_mx_pack
    assert g(P[0], 32, P[1], 2, 64, 64, P[2], P[3] + 1, None) == MISALIGNED
    assert g(P[0], 16, P[1], 2, 64, 64, P[2], P[3], None) == INVALID
    assert g(P[0], 32, P[1], 2, 64, 64, P[0], P[3], None) == ALIAS
    assert g(P[0], 32, P[1], 2, 64, 48, P[2], P[3], None) == UNSUPPORTED
    assert g(None, 0, None, 0, 0, 64, None, None, None) == OK


def mm(c=P[0], ldc=64, s=P[1], lds=16, fmt=1, wq=P[2], sc=P[3], b=None, y=P[4], dt=0, M=4, N=64, K=64):
    return mnb.mnb_mx_matmul(c, ldc, s, lds, fmt, wq, sc, b, y, dt, M, N, K, None)


def test_matmul_validation():
    assert mm(M=0, y=None) == OK and mm(N=0, y=None) == OK
    assert mm(M=-1) == INVALID and mm(fmt=5) == INVALID and mm(dt=2) == INVALID
    assert mm(K=40) == UNSUPPORTED and mm(K=1 << 25) == UNSUPPORTED and mm(M=1 << 30, N=1 << 30) == UNSUPPORTED
    assert mm(c=None) == INVALID and mm(wq=None) == INVALID and mm(y=None) == INVALID
    assert mm(ldc=48) == INVALID and mm(lds=8) == INVALID
    assert mm(ldc=72) == MISALIGNED and mm(y=P[4] + 2) == MISALIGNED and mm(b=P[5] + 2) == MISALIGNED
    for where in (P[0], P[1], P[2], P[3]):
        assert mm(y=where) == ALIAS
    assert mm(b=P[4] + 16) == ALIAS
    # a last row of a strided X that ends inside Y
    assert mm(y=P[0] + 3 * 4096 + 16, ldc=4096) == ALIAS
    assert mm(ldc=(1 << 23) + 16) == UNSUPPORTED and mm(lds=(1 << 23) + 16) == UNSUPPORTED


def norm(x=P[0], ldx=64, r=P[1], ldr=64, w=P[2], eps=1e-6, dt=0, M=4, K=64, h=P[3], ldh=64, y=P[4], ldy=64, fmt=0, c=None,
         ldc=0, s=None, lds=0):
    return mnb.mnb_rmsnorm(x, ldx, r, ldr, w, eps, dt, M, K, h, ldh, y, ldy, fmt, c, ldc, s, lds, None)


def test_rmsnorm_validation():
    mx = dict(fmt=1, c=P[5], ldc=64, s=P[6], lds=16)
    assert norm(M=0, x=None) == OK
    assert norm(M=-1) == INVALID and norm(dt=2) == INVALID and norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID
    assert norm(x=None) == INVALID and norm(w=None) == INVALID and norm(y=None) == INVALID
    assert norm(ldx=32) == INVALID and norm(ldr=32) == INVALID and norm(ldh=1) == INVALID and norm(ldy=63) == INVALID
    assert norm(x=P[0] + 1) == MISALIGNED and norm(w=P[2] + 1) == MISALIGNED
    assert norm(K=48, **mx) == UNSUPPORTED and norm(**dict(mx, fmt=7)) == INVALID and norm(**dict(mx, s=None)) == INVALID
    assert norm(x=P[0] + 2, **mx) == MISALIGNED and norm(ldh=66, **mx) == MISALIGNED and norm(**dict(mx, lds=20)) == MISALIGNED
    assert norm(**dict(mx, lds=0)) == INVALID
    # allowed in place: hidden = residual, hidden = x, y = x; refused: shifted or crossed overlaps
    assert norm(h=P[1] + 128) == ALIAS and norm(h=P[0], ldh=128) == ALIAS and norm(y=P[1]) == ALIAS and norm(y=P[3]) == ALIAS
    assert norm(h=P[2]) == ALIAS and norm(y=P[2]) == ALIAS and norm(y=P[0] + 2) == ALIAS
    assert norm(**dict(mx, c=P[0])) == ALIAS and norm(**dict(mx, s=P[5] + 16)) == ALIAS


def lp(x=P[0], dt=0, M=4, V=100, ldl=100, tok=P[1], top=0, o=P[2], e=P[3], tl=None, tt=None, ws=None, wsb=0):
    return mnb.mnb_logprobs(x, dt, M, V, ldl, tok, top, o, e, tl, tt, ws, wsb, None)


def test_logprobs_validation():
    t = dict(top=5, tl=P[4], tt=P[5])
    assert lp(M=0, x=None) == OK and lp(V=0, x=None) == OK
    assert lp(M=-1) == INVALID and lp(dt=3) == INVALID and lp(top=-1) == INVALID and lp(x=None) == INVALID
    assert lp(**dict(t, top=33)) == UNSUPPORTED and lp(V=(1 << 22) + 1, ldl=1 << 23) == UNSUPPORTED
    assert lp(V=4, **t) == INVALID                       # more alternatives than tokens
    assert lp(ldl=99) == INVALID and lp(o=None) == INVALID and lp(**dict(t, tl=None)) == INVALID
    assert lp(tok=None, e=None) == INVALID               # nothing to do
    assert lp(x=P[0] + 1) == MISALIGNED and lp(x=P[0] + 2, dt=2) == MISALIGNED and lp(tok=P[1] + 4) == MISALIGNED
    assert lp(e=P[3] + 2) == MISALIGNED and lp(**dict(t, tt=P[5] + 4)) == MISALIGNED
    assert lp(o=P[0] + 64) == ALIAS and lp(e=P[2]) == ALIAS and lp(**dict(t, tt=P[1])) == ALIAS
    assert mnb.mnb_logprobs_workspace_bytes(1, 49152, 0, 5) == 0     # one workgroup holds the row
    need = mnb.mnb_logprobs_workspace_bytes(1, 100000, 0, 5)
    assert need > 0
    a = dict(M=1, V=100000, ldl=100000)
    assert lp(**a, **t) == WORKSPACE and lp(ws=P[6], wsb=need - 1, **a, **t) == WORKSPACE
    assert lp(ws=P[0] + 16, wsb=need, **a, **t) == ALIAS and lp(ws=P[6] + 8, wsb=need, **a, **t) == MISALIGNED
    assert mnb.mnb_logprobs_workspace_bytes(0, 100, 0, 5) == 0 and mnb.mnb_logprobs_workspace_bytes(4, 100, 0, 40) == 0


# ------------------------------------------------------------------------------------------
# the torch binding's own checks (CPU tensors; every case fails before any library call)
# ------------------------------------------------------------------------------------------


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="on a GPU"):
        mnb.mx_quantize(x)
    with pytest.raises(TypeError):
        mnb.mx_quantize(x.double())
    with pytest.raises(ValueError, match="multiple of 32"):
        mnb.mx_quantize(x[:, :40])
    with pytest.raises(ValueError, match="contiguous"):
        mnb.mx_quantize(x.t())
    with pytest.raises(ValueError, match="2-D"):
        mnb.mx_quantize(x[0])
    with pytest.raises(ValueError, match="overlap"):
        mnb.mx_quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="format"):
        mnb.mx_quantize(x, 9)
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        mnb.mx_tensor(codes.int(), scales, mnb.MNB_MX_FP8)
    with pytest.raises(ValueError):
        mnb.mx_tensor(codes, scales[:, :1], mnb.MNB_MX_FP8)
    with pytest.raises(ValueError):
        mnb.mx_tensor(codes[:, :40], scales, mnb.MNB_MX_FP8)
    q = mnb.mx_tensor(codes, scales, mnb.MNB_MX_FP8)       # contiguous scales are laid out anew
    assert q.scales.stride(0) == 16 and q.K == 64 and torch.equal(q.scales, scales)
    assert mnb.mx_tensor(codes, q.scales, mnb.MNB_MX_FP8).scales is q.scales
    with pytest.raises(ValueError, match="apart"):
        mnb.mx_dequantize(mnb.MxTensor(codes, scales, mnb.MNB_MX_FP8))
    # one row: its 16 bytes must exist
    with pytest.raises(ValueError, match="apart"):
        mnb.mx_dequantize(mnb.MxTensor(codes[:1], scales[:1].clone(), mnb.MNB_MX_FP8))
    with pytest.raises(ValueError, match="MNB_MX_FP4"):
        mnb.mx_pack(q)
    w = mnb.MxWeight(torch.zeros(4096, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8), 64, 64)
    with pytest.raises(ValueError, match="on a GPU"):
        mnb.mx_matmul(q, w)
    with pytest.raises(ValueError, match="K="):
        mnb.mx_matmul(q, mnb.MxWeight(w.wq, w.sc, 64, 96))
    with pytest.raises(ValueError, match="packed codes"):
        mnb.mx_matmul(q, mnb.MxWeight(w.wq[:-16], w.sc, 64, 64))
    with pytest.raises(ValueError, match="out must"):
        mnb.mx_matmul(q, w, out=torch.zeros(4, 63, dtype=torch.float16))
    with pytest.raises(TypeError):
        mnb.mx_matmul(q, w, dtype=torch.float32)
    with pytest.raises(TypeError):
        mnb.mx_matmul(q, w, bias=torch.zeros(64))
    wn = torch.ones(64, dtype=torch.float16)
    with pytest.raises(TypeError):
        mnb.rmsnorm(x.float(), wn.float())
    with pytest.raises(TypeError):
        mnb.rmsnorm(x, wn.bfloat16())
    with pytest.raises(ValueError):
        mnb.rmsnorm(x, wn[:32])
    with pytest.raises(ValueError):
        mnb.rmsnorm(x, wn, residual=x[:2])
    with pytest.raises(ValueError, match="residual"):
        mnb.rmsnorm(x, wn, hidden=x)
    with pytest.raises(ValueError, match="multiple of 32"):
        mnb.rmsnorm(x[:, :40], wn[:40], fmt=mnb.MNB_MX_FP8)
    tok = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        mnb.logprobs(x, tok.int())
    with pytest.raises(ValueError):
        mnb.logprobs(x, tok[:3])
    with pytest.raises(ValueError, match="top"):
        mnb.logprobs(x, tok, top=33)
    with pytest.raises(ValueError, match="top"):
        mnb.logprobs(x[:, :3], tok, top=4)
    with pytest.raises(ValueError, match="columns"):
        mnb.logprobs(x[:, :0], tok)


# ------------------------------------------------------------------------------------------
# the references themselves
# ------------------------------------------------------------------------------------------


def test_reference_elements():
    codes = np.arange(256)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(codes), want, equal_nan=True)
    v = np.concatenate([np.linspace(-460, 460, 20001), np.ldexp(np.linspace(-1, 1, 4001), -5)])
    cast = torch.from_numpy(v.clip(-448, 448)).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_elements(v.astype(np.float32).astype(np.float64), 1), cast)
    # FP4: every value is its own nearest; ties go to the even code; beyond 6 stays 6
    assert np.array_equal(ref.round_elements(ref.FP4, 0), ref.FP4)
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9])
    assert np.array_equal(ref.round_elements(ties, 0), [0, 1, 1, 2, 2, 4, 4, 6])
    assert np.array_equal(ref.element_values(ref.element_codes(ref.FP4[None], 0), 0)[0], ref.FP4)


def test_reference_scales():
    x = np.zeros((1, 32 * 6))
    x[0, 32] = 4.0                # floor(log2) = 2
    x[0, 64] = 7.999
    x[0, 96] = np.inf
    x[0, 128] = 2.0 ** -130
    x[0, 160] = -3.0e38
    assert ref.block_scales(x, 0).tolist() == [[0, 127, 127, 255, 0, 127 + 127 - 2]]
    assert ref.block_scales(x, 1).tolist() == [[0, 121, 121, 255, 0, 127 + 127 - 8]]
    q, s = ref.quantize(x, 0)
    assert q[0, 64] == 6.0 and np.isnan(ref.dequantize(ref.element_codes(q, 0), s, 0)[0, 96:128]).all()


def test_reference_logprobs():
    x = np.array([[0.0, 1.0, 1.0, -np.inf], [2.0, 2.0, 2.0, 2.0]])
    l, h, _, v, i = ref.logprobs(x, np.array([1, 3]), 3)
    p = np.exp([0.0, 1.0, 1.0]) / np.exp([0.0, 1.0, 1.0]).sum()
    assert np.allclose(l, [np.log(p[1]), -np.log(4)]) and np.allclose(h, [-(p * np.log(p)).sum(), np.log(4)])
    assert i.tolist() == [[1, 2, 0], [0, 1, 2]] and np.allclose(v[1], -np.log(4))
