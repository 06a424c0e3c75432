"""Tensors that a call writes into count it, as torch's own in-place operations do, so that a graph that saved one for
its backward pass refuses to use it."""
from __future__ import annotations

import pytest

from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")


def inputs(M=5, K=64):
    x, r = torch.randn(M, K, device=DEV).half(), torch.randn(M, K, device=DEV).half()
    return x, r, torch.ones(K, device=DEV).half()


def test_written_tensors_count_it():
    x, r, w = inputs()
    before = [t._version for t in (x, r, w)]
    out, hidden = torch.empty_like(x), torch.empty_like(x)
    n = mnb.rmsnorm(x, w, residual=r, out=out, hidden=hidden)
    assert (out._version, hidden._version, n.y._version) == (1, 1, 1) and [t._version for t in (x, r, w)] == before
    mnb.rmsnorm(x, w, residual=r, hidden=r)
    assert r._version == before[1] + 1 and x._version == before[0]
    q = mnb.mx_quantize(x, mnb.MNB_MX_FP8)
    pw = mnb.mx_pack(mnb.mx_quantize(torch.randn(32, 64, device=DEV).half(), mnb.MNB_MX_FP4))
    v, y = torch.empty_like(x), torch.empty(5, 32, dtype=torch.float16, device=DEV)
    mnb.mx_dequantize(q, out=v)
    mnb.mx_matmul(q, pw, out=y)
    assert v._version == 1 and y._version == 1
    wide = torch.zeros(5, 128, dtype=torch.float16, device=DEV)      # a view counts for its base
    mnb.mx_dequantize(q, out=wide[:, :64])
    assert wide._version == 1


def test_a_saved_tensor_that_was_written_into_is_refused():
    x, r, w = inputs()
    a = torch.randn(5, 64, device=DEV).half().requires_grad_()
    y = (a * r).sum()
    mnb.rmsnorm(x, w, residual=r, hidden=r)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_are_written_into_anywhere():
    with torch.inference_mode():
        x, r, w = inputs()
        want = mnb.rmsnorm(x, w, residual=r)
        out = torch.empty_like(x)
        mnb.rmsnorm(x, w, residual=r, out=out)
    assert torch.equal(out, want.y)
    mnb.rmsnorm(x, w, residual=r, hidden=r, out=out)
    assert torch.equal(out, want.y) and torch.equal(r, want.hidden)
