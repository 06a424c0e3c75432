"""How far the product's sums are from exact ones, on rows whose results nearly cancel, so that the output shows the
sums' error and not its own rounding: each weight row carries blocks that take y out two bits at a time.

Bounds, of the sum of the magnitudes |x| |w| of a result:
  FP4 X  (K / 128 + 1) 2^-23: each instruction adds its 128 products and the running sum with an error of
         at most one unit of the last place of 32 bits of what it adds;
  FP8 X  2^-12, whatever the scales: the instruction's adder keeps fewer bits below its largest term."""
from __future__ import annotations

import numpy as np
import pytest

import _ops_ref as ref
from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")
FP4, FP8 = mnb.MNB_MX_FP4, mnb.MNB_MX_FP8
CANCEL = 12            # blocks that cancel


def to_mx(q, s, fmt):
    return mnb.mx_tensor(torch.from_numpy(ref.element_codes(q, fmt)).to(DEV), torch.from_numpy(s.astype(np.uint8)).to(DEV), fmt)


def values(q, s):
    return q * np.repeat(np.ldexp(1.0, s - 127), 32, 1)


def cancelling(r, N, K, fmt, spread):
    """One X row and N weight rows of K numbers and CANCEL blocks more, block scales over 2^-spread .. 2^spread."""
    def random(n, f):
        q, s = ref.quantize(r.standard_normal((n, K)), f)
        return q, s + r.integers(-spread, spread + 1, s.shape)
    (xq, xs), (wq, ws) = random(1, fmt), random(N, FP4)
    rest = -(values(xq, xs) @ values(wq, ws).T)[0]
    ones = np.zeros((1, 32 * CANCEL))
    ones[0, ::32] = 1.0
    cq, cs = np.zeros((N, 32 * CANCEL)), np.zeros((N, CANCEL), np.int64)
    for c in range(CANCEL):
        a = np.abs(rest)
        e = np.floor(np.log2(np.where(a > 0, a, 1.0))).astype(np.int64)
        m = np.where(a > 0, np.floor(np.ldexp(a, -e) * 2) / 2, 0.0)      # 1 or 1.5
        cq[:, 32 * c], cs[:, c] = np.copysign(m, rest), e + 127
        rest = rest - np.copysign(np.ldexp(m, e), rest)
    x = np.concatenate([xq, ones], 1), np.concatenate([xs, np.full((1, CANCEL), 127)], 1)
    return x, (np.concatenate([wq, cq], 1), np.concatenate([ws, cs], 1))


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("spread", [0, 1, 4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 500, 128), (7, 500, 2016), (32, 72, 9728), (40, 500, 480), (300, 500, 2016), (700, 4096, 2560)])
def test_sums_that_cancel(M, N, K, fmt, spread):
    r = np.random.default_rng([20261208, M, N, K, fmt, spread])
    x, w = cancelling(r, N, K, fmt, spread)
    xv, wv = values(*x), values(*w)
    want, size = (xv @ wv.T)[0], (np.abs(xv) @ np.abs(wv).T)[0]
    X = to_mx(np.repeat(x[0], M, 0), np.repeat(x[1], M, 0), fmt)
    got = mnb.mx_matmul(X, mnb.mx_pack(to_mx(*w, FP4)), dtype=torch.bfloat16).double().cpu().numpy()
    total = K + 32 * CANCEL
    bound = size * ((total / 128 + 1) * 2.0 ** -23 if fmt == FP4 else 2.0 ** -12) + np.abs(want) * 2.0 ** -8
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()
    assert (got == got[:1]).all()


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M", [1, 40])
def test_scales_at_the_ends_of_their_range(fmt, M):
    """Scale bytes from 0 (2^-127) to 254 (2^127) whose products lie inside 32 bits, each over a whole row and mixed in
    one.  The bounds above; results below the smallest normal number may be flushed."""
    r = np.random.default_rng([20261211, fmt, M])
    K, N = 256, 72
    pairs = [(0, 254), (254, 0), (0, 250), (1, 250), (127, 0), (0, 127), (127, 1), (3, 127), (20, 110), (0, 0), (64, 64), (240, 100), (253, 1), (200, 54)]
    mixed = np.array([0, 254, 127, 1, 250, 3, 200, 60])
    rows = [(np.full(K // 32, a), np.full(K // 32, b)) for a, b in pairs] + [(mixed, 254 - mixed)]
    for xs, ws in rows:
        xq, wq = ref.round_elements(r.uniform(-6, 6, (M, K)), fmt), ref.FP4[r.integers(0, 16, (N, K))]
        xs, ws = np.tile(xs, (M, 1)), np.tile(ws, (N, 1))
        each = np.ldexp(1.0, xs[:1] + ws[:1] - 254).repeat(32, 1)       # both scales of a term: in range where either alone is not
        want, size = (xq * each) @ wq.T, (np.abs(xq) * each) @ np.abs(wq).T
        got = mnb.mx_matmul(to_mx(xq, xs, fmt), mnb.mx_pack(to_mx(wq, ws, FP4)), dtype=torch.bfloat16).double().cpu().numpy()
        bound = size * ((K / 128 + 1) * 2.0 ** -23 if fmt == FP4 else 2.0 ** -12) + np.abs(want) * 2.0 ** -8 + 2.0 ** -126
        assert (np.abs(got - want) <= bound).all(), (xs[0, 0], ws[0, 0], (np.abs(got - want) / bound).max())
