"""The norm's MX codes against those of the norm in 64 bits, bit for bit, on rows whose outputs lie at
the borders of the element grid (ties, powers of two), where 32 bits alone take the wrong side.

Rows that lie at borders by construction have a mean square of exactly 1 (eps 0), so that y = h w: the
fillers below complete the sum of squares with powers of two.  32 bits lose the residuals that put them
to one side of it."""
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
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
# numbers below 2, whose block has its largest magnitude in [1, 2): elements are x / 2^-2 (FP4) or
# x / 2^-8 (FP8).  Ties that go up and ties that go down.
TIES = {FP4: [0.625, 1.25, 0.875, 0.4375, 0.1875], FP8: [1.0625, 1.3125, 1.1875, 1.4375, 0.59375]}
TOP = 1.5


def rng(*seed):
    return np.random.default_rng([20261207, *seed])


def dev(a, dt):
    return torch.from_numpy(np.asarray(a, np.float64)).to(dt).to(DEV)


def same_codes(q, want, fmt, where=""):
    v, s = ref.quantize(want, fmt)
    assert np.array_equal(q.scales.cpu().numpy(), s), where
    got, codes = q.codes.cpu().numpy(), ref.element_codes(v, fmt)
    assert np.array_equal(got, codes), (where, int((got != codes).sum()))


def block_of(ties, top):
    """32 numbers whose squares sum to 32 exactly: the ties, the largest, powers of two (but 2^-4, FP4's tie)."""
    b = [*ties, top]
    for v in [top, *(2.0 ** -e for e in range(12) if e != 4)]:
        while v * v <= 32 - np.square(b).sum():
            b.append(v)
    assert np.square(b).sum() == 32 and len(b) <= 32
    return np.array(b + [0.0] * (32 - len(b)))


def unit_row(fmt, K, r):
    """A row of mean square 1 with ties in every block: (numbers, mask of the ties)."""
    x = np.concatenate([block_of(TIES[fmt], TOP) for _ in range(K // 32)])
    tie = np.isin(x, TIES[fmt])
    for b in range(K // 32):
        at = r.permutation(32) + 32 * b
        x[32 * b:32 * b + 32], tie[32 * b:32 * b + 32] = x[at], tie[at]
    return x * r.choice([-1.0, 1.0], K), tie


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_random_rows_have_the_codes_of_the_64_bit_norm(dtype, fmt):
    for M, K in ((2000, 1024), (300, 4096), (40, 8192), (20, 36000), (1, 65536)):
        r = rng(1, fmt, M, K)
        x, res = dev(r.standard_normal((M, K)), DT[dtype]), dev(r.standard_normal((M, K)), DT[dtype])
        w = dev(1 + 0.2 * r.standard_normal(K), DT[dtype])
        X, R, W = (t.double().cpu().numpy() for t in (x, res, w))
        h = X + R
        want = h / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-6) * W
        n = mnb.rmsnorm(x, w, 1e-6, residual=res, fmt=fmt)
        same_codes(n.q, want, fmt, (M, K))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("K", [64, 2048, 4096, 8192, 40000])
def test_sums_past_32_bits_at_ties(dtype, fmt, K):
    """x at a tie, a residual too small for the 32-bit sum: y lies beside the tie by the residual's sign.
    The residuals' signs cancel in the sum of squares to second order (2^-48)."""
    r = rng(2, fmt, K)
    x, tie = unit_row(fmt, K, r)
    res = np.where(tie, 2.0 ** -24 * 2.0 ** np.floor(np.log2(np.abs(x) + (x == 0))), 0.0)
    if dtype == "fp16":
        res = np.where(tie, 2.0 ** -24, 0.0)                         # its smallest number
    sign = np.ones(K)
    for v in np.unique(np.abs(x[tie])):                              # half of each tie's up, half down
        at = np.flatnonzero(tie & (np.abs(x) == v))
        sign[at] = np.where(np.arange(len(at)) % 2 == 0, 1.0, -1.0) * np.sign(x[at])
    h = x + res * sign
    assert abs((h * h).mean() - 1) < 2.0 ** -44
    X, R = dev(np.stack([x, x]), DT[dtype]), dev(np.stack([res * sign, -res * sign]), DT[dtype])
    hh = np.stack([h, x - res * sign])
    n = mnb.rmsnorm(X, torch.ones(K, dtype=DT[dtype], device=DEV), 0.0, residual=R, fmt=fmt)
    same_codes(n.q, hh / np.sqrt((hh * hh).mean(-1, keepdims=True)), fmt)
    held = R.clone()                                                 # in place: the inputs are overwritten
    m = mnb.rmsnorm(X, torch.ones(K, dtype=DT[dtype], device=DEV), 0.0, residual=held, hidden=held, fmt=fmt)
    assert torch.equal(m.q.codes, n.q.codes) and torch.equal(m.q.scales, n.q.scales) and torch.equal(held, n.hidden)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("K", [64, 2048, 40000])
def test_the_norm_is_that_of_the_unrounded_sum(dtype, fmt, K):
    """The largest numbers carry a residual that a 32-bit sum loses, so the norm lies 2^-24 or so beside 1 and
    every tie to its side."""
    r = rng(3, fmt, K)
    x, tie = unit_row(fmt, K, r)
    big = np.abs(x) == TOP
    res = np.where(big, np.sign(x) * 2.0 ** -24, 0.0)
    h = np.stack([x + res, x - res])
    X, R = dev(np.stack([x, x]), DT[dtype]), dev(np.stack([res, -res]), DT[dtype])
    n = mnb.rmsnorm(X, torch.ones(K, dtype=DT[dtype], device=DEV), 0.0, residual=R, fmt=fmt)
    same_codes(n.q, h / np.sqrt((h * h).mean(-1, keepdims=True)), fmt)


def within_half_a_step(got, want, dt, K):
    """One rounding of `dt` beside the 32-bit steps (the sum of squares and the root are in 64 bits): 2^-21."""
    top, least = torch.finfo(dt).max, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    g = got.double().cpu().numpy()
    over = np.abs(want) >= top * (1 + torch.finfo(dt).eps / 4)
    assert (np.abs(g[over]) == np.inf).all() and (np.sign(g[over]) == np.sign(want[over])).all()
    err = np.abs(g[~over] - want[~over])
    assert (err <= np.abs(want[~over]) * (torch.finfo(dt).eps / 2 + 2.0 ** -21) + least / 2).all(), err.max()


@pytest.mark.parametrize("K", [64, 577, 2048, 4096, 8192, 9000, 40000])
def test_rows_whose_norm_is_near_the_ends_of_32_bits(K):
    """bfloat16 rows of subnormals with eps 0 (the root's inverse is past 32 bits), rows near the largest number (it
    is subnormal), and sums past the largest 32-bit number: y is of order 1 in all of them."""
    r = rng(4, K)
    dt = torch.bfloat16
    x = np.stack([r.integers(1, 9, K) * 2.0 ** -133 * r.choice([-1.0, 1.0], K),
                  r.uniform(0.5, 1, K) * 3.3e38 * r.choice([-1.0, 1.0], K),
                  r.uniform(0.5, 1, K) * 2e38,
                  r.standard_normal(K) * 1e-36,
                  r.standard_normal(K) * 2.0 ** 100,
                  r.standard_normal(K)])
    res = np.stack([r.integers(1, 9, K) * 2.0 ** -133, np.zeros(K), r.uniform(0.5, 1, K) * 2.5e38, np.zeros(K),
                    r.standard_normal(K) * 2.0 ** 100, r.standard_normal(K)])
    X, R, W = dev(x, dt), dev(res, dt), dev(1 + 0.2 * r.standard_normal(K), dt)
    x, res, w = (t.double().cpu().numpy() for t in (X, R, W))
    for residual in (None, R):
        h = x if residual is None else x + res
        want = h / np.sqrt((h * h).mean(-1, keepdims=True)) * w
        n = mnb.rmsnorm(X, W, 0.0, residual=residual)
        within_half_a_step(n.y, want, dt, K)
        if residual is not None:
            within_half_a_step(n.hidden, h, dt, K)
        if K % 32 == 0:
            for fmt in (FP4, FP8):
                n = mnb.rmsnorm(X, W, 0.0, residual=residual, fmt=fmt, keep16=True)
                within_half_a_step(n.y, want, dt, K)
                same_codes(n.q, want, fmt, K)


# 32 whole numbers whose squares sum to 32 * 128^2
IN_128THS = np.array([192, 191, 191, 160, 160, 150, 150, 150, 150, 131, 131, 131, 131, 131, 131, 129, 129, 129, 127, 125, 125, 125, 125, 113, 113, 80, 65, 65, 33, 13, 7, 7])


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("K", [64, 2048, 40000])
def test_outputs_among_the_smallest_numbers(fmt, K):
    """Weights of 2^-130 and less: the block's scale is the smallest, FP8's ties odd multiples of 2^-137, and 32
    bits hold y in steps of 2^-149.  Residuals that such steps lose put y beside the tie."""
    r = rng(5, fmt, K)
    x = np.tile(IN_128THS / 128, K // 32)                # mean square 1, half of them odd
    res = np.where(x > 0, 2.0 ** -22, 0.0)
    sign = np.ones(K)
    for v in np.unique(x):
        at = np.flatnonzero(x == v)
        sign[at] = np.where(np.arange(len(at)) % 2 == 0, 1.0, -1.0)
    h = np.stack([x + res * sign, x - res * sign])
    X, R = dev(np.stack([x, x]), torch.bfloat16), dev(np.stack([res * sign, -res * sign]), torch.bfloat16)
    for e in (-125, -127, -128, -129, -130, -131, -132, -133):
        W = dev(np.full(K, 2.0 ** e), torch.bfloat16)
        want = h / np.sqrt((h * h).mean(-1, keepdims=True)) * 2.0 ** e
        n = mnb.rmsnorm(X, W, 0.0, residual=R, fmt=fmt, keep16=True)
        same_codes(n.q, want, fmt, e)
        y = n.y.double().cpu().numpy()
        assert (np.abs(y - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -134).all()
