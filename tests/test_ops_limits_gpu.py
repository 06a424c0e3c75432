"""Calls of more outputs than one part of a launch's index range held."""
from __future__ import annotations

import numpy as np
import pytest

import _ops_ref as ref
from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("fmt", [mnb.MNB_MX_FP4, mnb.MNB_MX_FP8])
def test_product_of_more_than_2_to_32_outputs(fmt):
    """131077 x 49152 results: 64 rows of X repeat, and so do Y's."""
    M, N, K = 131077, 49152, 64
    r = np.random.default_rng([20261209, fmt])
    (xq, xs), (wq, ws) = (ref.quantize(r.integers(-6, 7, (n, K)) / 2.0, f) for n, f in ((64, fmt), (N, mnb.MNB_MX_FP4)))
    def to_mx(q, s, f):
        return mnb.mx_tensor(torch.from_numpy(ref.element_codes(q, f)).to(DEV), torch.from_numpy(s.astype(np.uint8)).to(DEV), f)
    w = mnb.mx_pack(to_mx(wq, ws, mnb.MNB_MX_FP4))
    x = to_mx(xq, xs, fmt)
    want = mnb.mx_matmul(x, w)
    xv, wv = (torch.from_numpy(q * np.repeat(np.ldexp(1.0, s - 127), 32, 1)).to(DEV) for q, s in ((xq, xs), (wq, ws)))
    assert torch.equal(want, (xv @ wv.t().contiguous()).half())
    rep = -(-M // 64)
    y = mnb.mx_matmul(mnb.mx_tensor(x.codes.repeat(rep, 1)[:M], x.scales.repeat(rep, 1)[:M], fmt), w)
    for at in range(0, M, 16384):
        part = y[at:at + 16384]
        full = part[:len(part) // 64 * 64].view(-1, 64, N)
        assert bool((full == want).all()) and torch.equal(part[len(full) * 64:], want[:len(part) % 64]), at


@pytest.mark.parametrize("M,V,top", [((1 << 22) + 5, 8, 3), ((1 << 22) - 1, 5, 5), (9 << 20, 3, 0)])
def test_logprobs_of_more_than_2_to_22_rows(M, V, top):
    """1000 rows repeat, and so do their results."""
    r = np.random.default_rng([20261210, M])
    x = torch.from_numpy(r.standard_normal((1000, V))).to(DEV).half()
    tok = torch.from_numpy(r.integers(0, V, 1000)).to(DEV)
    want = mnb.logprobs(x, tok, top)
    rep = -(-M // 1000)
    got = mnb.logprobs(x.repeat(rep, 1)[:M], tok.repeat(rep)[:M], top)
    for a, b in zip(got, want):
        if b is not None:
            assert a.shape[0] == M and torch.equal(a, b.repeat(rep, *[1] * (b.dim() - 1))[:M])
