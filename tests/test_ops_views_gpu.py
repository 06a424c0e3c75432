"""Tensors whose rows lie between each other's rows in one buffer, without sharing a byte."""
from __future__ import annotations

import pytest

from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")


def halves(M, K, dtype=torch.float16, pad=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wide = torch.randn(M, 2 * K + pad, generator=g, device=DEV).to(dtype)
    return wide, wide[:, :K], wide[:, K:2 * K]


@pytest.mark.parametrize("M,K,pad", [(1, 64, 0), (7, 576, 32), (40, 577, 1), (33, 20000, 0)])
def test_norm_into_the_columns_beside_its_input(M, K, pad):
    w = torch.rand(K, device=DEV).half() + 0.5
    wide, x, y = halves(M, K, pad=pad)
    want, tail = mnb.rmsnorm(x.clone(), w).y, wide[:, 2 * K:].clone()
    got = mnb.rmsnorm(x, w, out=y)
    assert got.y.data_ptr() == y.data_ptr() and torch.equal(y, want) and torch.equal(wide[:, 2 * K:], tail)
    # x, residual, hidden and y as four column ranges of one buffer, y and hidden in either order
    four = torch.randn(M, 4 * K, device=DEV).half()
    a, b, c, d = (four[:, i * K:(i + 1) * K] for i in range(4))
    want = mnb.rmsnorm(a.clone(), w, residual=b.clone())
    for hidden, out in ((c, d), (d, c)):
        got = mnb.rmsnorm(a, w, residual=b, hidden=hidden, out=out)
        assert torch.equal(got.y, want.y) and torch.equal(got.hidden, want.hidden)
    got = mnb.rmsnorm(a, w, residual=b, hidden=b, out=c)          # in place, beside another output
    assert torch.equal(c, want.y) and torch.equal(b, want.hidden)


def test_columns_that_do_share_bytes_are_refused():
    M, K = 9, 64
    w = torch.ones(K, device=DEV).half()
    wide, x, _ = halves(M, K)
    before = wide.clone()
    for shift in (1, 32, K - 1):
        with pytest.raises(RuntimeError, match="ALIAS"):
            mnb.rmsnorm(x, w, out=wide[:, shift:shift + K])
    with pytest.raises(RuntimeError, match="ALIAS"):
        mnb.rmsnorm(wide[:, K:], w, out=wide[:, K // 2:K // 2 + K])
    flat = wide.view(-1)
    with pytest.raises(RuntimeError, match="ALIAS"):               # the end of each row of one, the start of the next of the other
        mnb.rmsnorm(x[:-1], w, out=flat[K + 32:].as_strided((M - 1, K), (2 * K, 1)))
    with pytest.raises(RuntimeError, match="ALIAS"):               # other row distances
        mnb.rmsnorm(x[:3], w, out=flat[K:K + 3 * 3 * K].view(3, 3 * K)[:, :K])
    assert torch.equal(wide, before)


@pytest.mark.parametrize("fmt", [mnb.MNB_MX_FP4, mnb.MNB_MX_FP8])
def test_dequantised_beside_the_codes(fmt):
    """Codes and their values as columns of one buffer of bytes."""
    M, K = 50, 128
    row = K if fmt == mnb.MNB_MX_FP8 else K // 2
    wide = torch.zeros(M, row + 2 * K, dtype=torch.uint8, device=DEV)
    q = mnb.mx_quantize(torch.randn(M, K, device=DEV).half(), fmt)
    wide[:, :row] = q.codes
    held = mnb.mx_tensor(wide[:, :row], q.scales, fmt)
    out = wide.view(torch.float16)[:, row // 2:]
    got = mnb.mx_dequantize(held, torch.float16, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, mnb.mx_dequantize(q)) and torch.equal(wide[:, :row], q.codes)
