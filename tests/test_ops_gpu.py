"""GPU results of the operators in include/mnb_ops.h against plain 64-bit references.

Tolerances (each derived beside its test): quantisation, packing, dequantisation and products
whose sums are exact in 32 bits are compared bit for bit; rounded outputs by half a step of
their type plus the 32-bit errors of the sums behind them.
"""
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
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def rng(*seed):
    return np.random.default_rng([20261206, *seed])


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def rounded(a, dtype):
    """float64 values rounded to a torch type, as float64 (through 32 bits: the inputs have no more)."""
    return torch.from_numpy(np.asarray(a, np.float64)).to(torch.float32).to(dtype).double().numpy()


def to_mx(q, s, fmt):
    """Device MxTensor of element values and scale bytes."""
    return mnb.mx_tensor(dev(ref.element_codes(q, fmt)), dev(s.astype(np.uint8)), fmt)


def strided(t, extra, fill=7.0):
    """The same values as rows of a wider tensor."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ------------------------------------------------------------------------------------------
# quantisation: bit for bit
# ------------------------------------------------------------------------------------------


def check_quantize(x, fmt):
    q = mnb.mx_quantize(x, fmt)
    want, scales = ref.quantize(f64(x), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), ref.element_codes(want, fmt))
    return q


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (7, 576), (64, 2048), (1000, 160), (5, 4128)])
def test_quantize(fmt, dtype, M, K):
    r = rng(1, fmt, M, K)
    x = dev(r.standard_normal((M, K)) * np.exp(2 * r.standard_normal((M, 1)))).to(DT[dtype])
    check_quantize(x, fmt)
    check_quantize(strided(x, 64), fmt)


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_quantize_special_blocks(fmt, dtype):
    t = DT[dtype]
    tiny, huge = torch.finfo(t).smallest_normal, torch.finfo(t).max
    x = torch.zeros(4, 32 * 10, dtype=torch.float64)
    x[0, 33] = float("inf")
    x[0, 64] = float("nan")
    x[0, 100] = float("-inf")
    x[1, :32] = torch.linspace(-huge, huge, 32, dtype=torch.float64)
    x[1, 32:64] = torch.linspace(0, tiny, 32, dtype=torch.float64)          # subnormals
    x[1, 64] = torch.finfo(t).smallest_normal * torch.finfo(t).eps          # the smallest number alone
    x[2, :32] = -0.0
    # every tie of either format, scaled by powers of two
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, 4.25, 6.5, -.25, -.75, -1.25, -2.5, -5, 4], dtype=torch.float64)
    for b in range(6):
        x[3, 32 * b:32 * b + 16] = ties * 2.0 ** (b - 3)
    x[3, 192:224] = 256 + 16 * torch.arange(32, dtype=torch.float64) / 2    # E4M3 ties and the clamp from 448 on
    check_quantize(x.to(t).to(DEV), fmt)


def test_quantize_every_half():
    """All finite binary16 numbers, each alone in its block."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).view(np.float16)
    bits = bits[np.isfinite(bits)]
    x = torch.zeros(len(bits), 32, dtype=torch.float16)
    x[:, 5] = torch.from_numpy(bits.copy())
    for fmt in (FP4, FP8):
        check_quantize(x.to(DEV), fmt)


@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_dequantize(fmt):
    """All codes under scales from the smallest to NaN, bit for bit in every type."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 2 if fmt == FP4 else 1))
    K = codes.shape[1] * (2 if fmt == FP4 else 1)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // 32, 1)
    t = mnb.mx_tensor(dev(codes), dev(scales), fmt)
    want = torch.from_numpy(ref.dequantize(codes, scales, fmt))
    for name, dt in DT.items():
        got = mnb.mx_dequantize(t, dt).cpu()
        w = want.to(torch.float32).to(dt)          # exact in 32 bits but for overflow, then one rounding
        assert torch.equal(torch.nan_to_num(got.float(), nan=12345.0), torch.nan_to_num(w.float(), nan=12345.0)), name
    wide = torch.full((256, K + 32), 3.0, dtype=torch.float16, device=DEV)
    mnb.mx_dequantize(t, torch.float16, out=wide[:, :K])
    assert bool((wide[:, K:] == 3.0).all()) and torch.equal(wide[:, :K].view(torch.int16), mnb.mx_dequantize(t).view(torch.int16))


@pytest.mark.parametrize("N,K", [(1, 32), (64, 128), (65, 96), (130, 1056), (1000, 576)])
def test_pack_layout(N, K):
    r = rng(2, N, K)
    codes, scales = r.integers(0, 256, (N, K // 2), dtype=np.uint8), r.integers(0, 256, (N, K // 32), dtype=np.uint8)
    w = mnb.mx_pack(mnb.mx_tensor(dev(codes), dev(scales), FP4))
    wq, sc = ref.pack(codes, scales, N, K)
    assert np.array_equal(w.wq.cpu().numpy(), wq) and np.array_equal(w.sc.cpu().numpy(), sc)


# ------------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------------

SHAPES = [(1, 1, 32), (1, 64, 128), (1, 896, 896), (1, 1000, 4096), (2, 65, 96), (5, 200, 576), (8, 1000, 640), (16, 130, 1056),
          (16, 3000, 512), (17, 64, 32), (17, 65, 160), (20, 3000, 512), (32, 1000, 1056), (33, 64, 32), (34, 65, 160), (33, 72, 576), (64, 320, 512), (100, 130, 1056), (128, 128, 2048),
          (129, 257, 320), (256, 512, 4096), (300, 1000, 800), (513, 136, 96)]


def exact_operands(r, M, N, K, fmt):
    """Operands whose every partial sum is a multiple of 2^-4 below 2^20 in magnitude for K <= 4096
    (|x| <= 6 * 2, |w| <= 6 * 2, quanta 1/4 each): exact in 32 bits in any order."""
    def values(n, f):
        codes = r.integers(0, 16, (n, K))
        q = ref.FP4[codes] if f == FP4 else np.where(r.random((n, K)) < .5, ref.FP4[codes], np.rint(r.uniform(-6, 6, (n, K))))
        return q, r.integers(126, 129, (n, K // 32))
    return values(M, fmt), values(N, FP4)


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_exact_sums(M, N, K, fmt):
    r = rng(3, M, N, K, fmt)
    (xq, xs), (wq, ws) = exact_operands(r, M, N, K, fmt)
    want = (xq * np.repeat(np.ldexp(1.0, xs - 127), 32, 1)) @ (wq * np.repeat(np.ldexp(1.0, ws - 127), 32, 1)).T
    x, w = to_mx(xq, xs, fmt), mnb.mx_pack(to_mx(wq, ws, FP4))
    for dt in (torch.float16, torch.bfloat16):
        if dt == torch.float16 and np.abs(want).max() > 60000:
            continue
        got = f64(mnb.mx_matmul(x, w, dtype=dt))
        assert np.array_equal(got, rounded(want, dt)), (M, N, K, fmt, dt)
    bias = rounded(r.integers(-8, 9, N) / 4.0, torch.bfloat16)
    got = f64(mnb.mx_matmul(x, w, bias=dev(bias, torch.bfloat16), dtype=torch.bfloat16))
    assert np.array_equal(got, rounded(want + bias, torch.bfloat16))


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M,N,K", [(4097, 4100, 416), (2100, 9000, 1120), (4352, 4096, 8864), (1000, 2100, 8864), (40, 300, 17056),
                                   (64, 260, 16800), (900, 4000, 4448), (900, 4032, 4448), (1020, 4090, 2080), (100, 131, 2080), (333, 1000, 1568), (65, 2560, 9728),
                                   (32, 8190, 2048), (32, 49100, 576), (21, 41000, 2112), (30, 65600, 576), (17, 131100, 1056), (24, 12300, 4128)])
def test_matmul_exact_sums_large(M, N, K, fmt):
    """Tiles of every height, K past one panel of scales and ending inside a step; the reference is
    a 64-bit product on the GPU.  Partial sums here stay below 2^18 (they are random walks of at
    most 17056 terms up to 144), multiples of 2^-4: exact in 32 bits."""
    r = rng(17, M, N, K, fmt)
    (xq, xs), (wq, ws) = exact_operands(r, M, N, K, fmt)
    x, w = to_mx(xq, xs, fmt), mnb.mx_pack(to_mx(wq, ws, FP4))
    xv = dev(xq) * dev(np.ldexp(1.0, xs - 127)).repeat_interleave(32, 1)
    wv = dev(wq) * dev(np.ldexp(1.0, ws - 127)).repeat_interleave(32, 1)
    want = xv @ wv.t().contiguous()
    for dt in (torch.float16, torch.bfloat16):
        assert torch.equal(mnb.mx_matmul(x, w, dtype=dt), want.float().to(dt)), dt


def random_mx(r, n, K, fmt, spread=1.0):
    q, s = ref.quantize(r.standard_normal((n, K)) * np.exp(spread * r.standard_normal((n, K // 32))).repeat(32, 1), fmt)
    return q, s


def product_bound(x, w, y, K, dt):
    """Half a step of the output, and of the sums: every 128-k instruction adds its exact
    products to the running sum with an error of at most 2^-12 of their largest magnitudes'
    sum (the adder keeps fewer than 24 bits below its largest term when one operand is FP8;
    FP4 sums are far closer), 2^-23 for each addition to the running sum."""
    absum = np.abs(x) @ np.abs(w).T
    return np.abs(y) * torch.finfo(dt).eps / 2 * 1.01 + absum * (2.0 ** -12 + K / 128 * 2.0 ** -23) + 2.0 ** -24


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 2048), (1, 130, 16384), (8, 4096, 576), (16, 896, 896), (40, 300, 2560), (1024, 512, 4096)])
def test_matmul_random(M, N, K, fmt):
    r = rng(4, M, N, K, fmt)
    (xq, xs), (wq, ws) = random_mx(r, M, K, fmt), random_mx(r, N, K, FP4, 0.3)
    xv, wv = xq * np.repeat(ref.scale_values(xs), 32, 1), wq * np.repeat(ref.scale_values(ws), 32, 1)
    want = xv @ wv.T
    for dt in (torch.float16, torch.bfloat16):
        scale = 1.0 if np.abs(want).max() < 6e4 else None
        if scale is None and dt == torch.float16:
            continue
        got = f64(mnb.mx_matmul(to_mx(xq, xs, fmt), mnb.mx_pack(to_mx(wq, ws, FP4)), dtype=dt))
        err = np.abs(got - want)
        assert (err <= product_bound(xv, wv, want, K, dt)).all(), (err / product_bound(xv, wv, want, K, dt)).max()
        # as a whole the rounding of the output dominates: uniform, 1 / sqrt(3) of half a step at most
        assert np.linalg.norm(err) <= np.linalg.norm(want) * torch.finfo(dt).eps / 2


@pytest.mark.parametrize("M", [4, 40])
def test_matmul_nan_stays_in_its_row_and_column(M):
    r = rng(5, M)
    N, K = 200, 416                                  # ends inside a step and inside a scale dword
    (xq, xs), (wq, ws) = exact_operands(r, M, N, K, FP8)
    clean = f64(mnb.mx_matmul(to_mx(xq, xs, FP8), mnb.mx_pack(to_mx(wq, ws, FP4))))
    xs2, ws2 = xs.copy(), ws.copy()
    xs2[1, 12] = 255
    ws2[70, 3] = 255
    x = to_mx(xq, xs2, FP8)
    x.codes[2, 400] = 0x7F                           # a NaN element
    got = f64(mnb.mx_matmul(x, mnb.mx_pack(to_mx(wq, ws2, FP4))))
    bad = np.zeros((M, N), bool)
    bad[[1, 2]] = True
    bad[:, 70] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("M", [3, 50])
def test_matmul_ignores_bytes_past_k(M):
    """Bytes between a row's scales and its next, and behind its codes, may hold anything, and
    nothing behind the output's rows is written."""
    r = rng(6, M)
    for fmt in (FP4, FP8):
        N, K = 72, 160
        (xq, xs), (wq, ws) = exact_operands(r, M, N, K, fmt)
        w = mnb.mx_pack(to_mx(wq, ws, FP4))
        x = to_mx(xq, xs, fmt)
        want = mnb.mx_matmul(x, w)
        codes = torch.full((M, x.codes.shape[1] + 48), 0x7F, dtype=torch.uint8, device=DEV)
        scales = torch.full((M, 48), 255, dtype=torch.uint8, device=DEV)
        codes[:, :x.codes.shape[1]], scales[:, :K // 32] = x.codes, x.scales
        x2 = mnb.mx_tensor(codes[:, :x.codes.shape[1]], scales[:, :K // 32], fmt)
        assert x2.scales.data_ptr() == scales.data_ptr()
        out = torch.full((M + 8, N), 5.0, dtype=torch.float16, device=DEV)
        got = mnb.mx_matmul(x2, w, out=out[:M])
        assert torch.equal(got, want) and bool((out[M:] == 5.0).all())


def test_matmul_empty():
    w = mnb.mx_pack(to_mx(np.zeros((64, 64)), np.full((64, 2), 127), FP4))
    x = to_mx(np.zeros((3, 64)), np.full((3, 2), 127), FP8)
    empty = mnb.MxTensor(x.codes[:0], x.scales[:0], FP8)
    assert mnb.mx_matmul(empty, w).shape == (0, 64)
    none = mnb.mx_quantize(torch.zeros(3, 0, dtype=torch.float16, device=DEV), FP8)
    wn = mnb.mx_pack(mnb.mx_quantize(torch.zeros(64, 0, dtype=torch.float16, device=DEV), FP4))
    bias = torch.arange(64, device=DEV).half()
    assert torch.equal(mnb.mx_matmul(none, wn, bias=bias), bias.expand(3, 64))
    assert bool((mnb.mx_matmul(none, wn) == 0).all())
    assert bool((mnb.mx_matmul(x, w) == 0).all())


# ------------------------------------------------------------------------------------------
# norm
# ------------------------------------------------------------------------------------------


def norm_inputs(r, M, K, dt, residual):
    x = rounded(r.standard_normal((M, K)) * np.exp(0.5 * r.standard_normal(K)), dt)
    res = rounded(r.standard_normal((M, K)), dt) if residual else None
    return x, res, rounded(1 + 0.2 * r.standard_normal(K), dt)


def check16(got, want, dt, K):
    """Half a step of the output; the sum of squares has at most K / 64 + 16 additions in line for
    K <= 65536, each 2^-24, halved by the root, and four more roundings follow; plus half the
    smallest subnormal."""
    rel = torch.finfo(dt).eps / 2 + (K / 64 + 24) * 2.0 ** -24
    assert (np.abs(f64(got) - want) <= np.abs(want) * rel + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2).all()


def check_mx(q, want, fmt, K):
    """The quantised output of values within (K / 64 + 24) 2^-24 of `want`: blocks whose scale is the
    same at both ends of that interval have elements between the ends' own."""
    d = (K / 64 + 24) * 2.0 ** -24
    (lo, sl), (hi, sh) = ref.quantize(want * (1 - d), fmt), ref.quantize(want * (1 + d), fmt)
    s = q.scales.cpu().numpy()
    got = ref.element_values(q.codes.cpu().numpy(), fmt)
    sure = sl == sh
    assert sure.mean() > 0.99 or (~sure).sum() <= 2
    assert (s[sure] == sl[sure]).all()
    el = np.repeat(sure, 32, -1)
    a, lo, hi = np.abs(got)[el], np.abs(lo)[el], np.abs(hi)[el]
    assert (a >= lo).all() and (a <= hi).all() and (np.sign(got)[el] * np.sign(want)[el] >= 0).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (1, 32), (5, 64), (33, 576), (4, 896), (2, 1001), (1, 2048), (70, 2056), (9, 4096),
                                 (3, 5120), (2, 8192), (2, 8224), (2, 16384), (1, 40000), (1, 65536)])
def test_rmsnorm(dtype, M, K):
    dt = DT[dtype]
    x, res, w = norm_inputs(rng(7, M, K), M, K, dt, True)
    X, R, W = dev(x, dt), dev(res, dt), dev(w, dt)
    want, h = ref.rmsnorm(x, res, w, 1e-6)
    plain = ref.rmsnorm(x, None, w, 1e-5)[0]
    n = mnb.rmsnorm(X, W, 1e-6, residual=R)
    check16(n.y, want, dt, K)
    # the 32-bit sum, itself within 2^-24, then half a step
    assert (np.abs(f64(n.hidden) - h) <= np.abs(h) * (torch.finfo(dt).eps / 2 + 2.0 ** -23) + 2.0 ** -25).all()
    n = mnb.rmsnorm(X, W, 1e-5)
    assert n.hidden is None and n.q is None
    check16(n.y, plain, dt, K)
    # strided rows, outputs into wider tensors, unaligned views
    wide = torch.full((M, K + 5), 9.0, dtype=dt, device=DEV)
    n = mnb.rmsnorm(strided(X, 3), W, 1e-6, residual=strided(R, 9), out=wide[:, 2:K + 2])
    check16(n.y, want, dt, K)
    assert bool((wide[:, :2] == 9).all()) and bool((wide[:, K + 2:] == 9).all())
    if K % 32 == 0:
        for fmt in (FP4, FP8):
            n = mnb.rmsnorm(X, W, 1e-6, residual=R, fmt=fmt, keep16=True)
            check_mx(n.q, want, fmt, K)
            check16(n.y, want, dt, K)
            assert (np.abs(f64(n.hidden) - h) <= np.abs(h) * (torch.finfo(dt).eps / 2 + 2.0 ** -23) + 2.0 ** -25).all()
            n = mnb.rmsnorm(X, W, 1e-5, fmt=fmt)
            assert n.y is None and n.hidden is None
            check_mx(n.q, plain, fmt, K)


def test_rmsnorm_in_place():
    for K in (576, 577, 20000):
        x, res, w = norm_inputs(rng(8, K), 5, K, torch.float16, True)
        X, R, W = dev(x, torch.float16), dev(res, torch.float16), dev(w, torch.float16)
        want = mnb.rmsnorm(X, W, residual=R)
        r2 = R.clone()
        n = mnb.rmsnorm(X, W, residual=r2, hidden=r2)
        assert torch.equal(r2, want.hidden) and torch.equal(n.y, want.y)
        x2 = X.clone()
        n = mnb.rmsnorm(x2, W, residual=R, hidden=x2)
        assert torch.equal(x2, want.hidden) and torch.equal(n.y, want.y)
        x3 = X.clone()
        n = mnb.rmsnorm(x3, W, residual=R, out=x3)
        assert torch.equal(x3, want.y) and torch.equal(n.hidden, want.hidden)
        with pytest.raises(RuntimeError, match="ALIAS"):
            mnb.rmsnorm(X, W, residual=R, out=R)


def test_rmsnorm_special_rows():
    """Rows of zeros, with infinities and NaN, large and tiny values: each row alone."""
    K = 640
    x = torch.zeros(6, K, dtype=torch.bfloat16)
    x[1] = 1e-30
    x[2] = 3e18                                   # squares near the top of 32 bits
    x[3] = 1.0
    x[3, 5] = float("nan")
    x[4] = 1.0
    x[4, 7] = float("inf")
    x[5] = torch.linspace(-1, 1, K)
    W = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    for fmt in (None, FP4, FP8):
        n = mnb.rmsnorm(x.to(DEV), W, 1e-6, fmt=fmt, keep16=True)
        y = f64(n.y)
        want = ref.rmsnorm(f64(x[[0, 1, 5]]), None, np.ones(K), 1e-6)[0]
        check16(n.y[[0, 1, 5]], want, torch.bfloat16, K)
        assert np.abs(y[2] - 1).max() < 0.01 and np.isnan(y[3]).all()
        assert np.isnan(y[4, 7]) and (np.delete(y[4], 7) == 0).all()
        if fmt is not None:
            s = n.q.scales.cpu().numpy()
            assert (s[0] == 0).all() and (s[3] == 255).all() and s[4, 0] == 255 and (s[4, 1:] == 0).all()


# ------------------------------------------------------------------------------------------
# log probabilities
# ------------------------------------------------------------------------------------------


def check_logprobs(x, dt, tokens, top, got=None):
    """32-bit errors: S and T are sums of terms each within 2^-22 (exp2 and its argument, weighted
    by the term, at most |d| 1.5 * 2^-24 more), added in at most 96 steps of 2^-24; the final differences
    round at the size of their operands."""
    v = f64(x)
    lp, ent, spread, tv, ti = ref.logprobs(v, tokens, top)
    got = got or mnb.logprobs(x, dev(tokens), top)
    sum_rel = 100 * 2.0 ** -24 + spread * 1.5 * 2.0 ** -24
    size = np.abs(lp) + np.abs(v.max(-1)) * 0 + np.log(v.shape[1]) + 1
    assert (np.abs(f64(got.logprob) - lp) <= sum_rel + size * 2.0 ** -23).all()
    assert (np.abs(f64(got.entropy) - ent) <= sum_rel * (1 + 2 * spread) + (np.abs(ent) + spread + 1) * 2.0 ** -23).all()
    if top:
        assert np.array_equal(got.top_tokens.cpu().numpy(), ti)
        assert (np.abs(f64(got.top_logprobs) - tv) <= sum_rel[:, None] + (np.abs(tv) + size[:, None]) * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (3, 2, 2), (2, 31, 20), (5, 33, 32), (1, 500, 5), (4, 2041, 32), (3, 4088, 20),
                                     (1, 4097, 8), (2, 16376, 3), (1, 49152, 5), (2, 50257, 20), (3, 57337, 32), (2, 49153, 5), (1, 98305, 9), (2, 147456, 32), (1, 262144, 32),
                                     (300, 1000, 20), (260, 49152, 32), (1100, 2100, 1), (2, 131072, 0), (1, 1000003, 7)])
def test_logprobs(dtype, M, V, top):
    r = rng(9, M, V, top)
    x = r.standard_normal((M, V)) * 3
    x[np.arange(M), r.integers(0, V, M)] += 8
    check_logprobs(dev(x).to(DT[dtype]), DT[dtype], r.integers(0, V, M), top)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("V", [1001, 49153])
def test_logprobs_unaligned_rows(dtype, V):
    r = rng(10, V)
    M = 5
    flat = dev(r.standard_normal(M * (V + 3) + 8)).to(DT[dtype])
    for at in range(8):
        x = flat[at:at + M * (V + 3)].view(M, V + 3)[:, :V]
        check_logprobs(x, DT[dtype], r.integers(0, V, M), 9)


@pytest.mark.parametrize("M,V", [(2, 700), (1, 49152), (300, 49152), (257, 3000)])
def test_logprobs_ties(M, V):
    """Equal logits come in index order, whole rows of them, the two zeros alike."""
    r = rng(11, M, V)
    tok = r.integers(0, V, M)
    check_logprobs(torch.zeros(M, V, dtype=torch.float16, device=DEV), None, tok, 32)
    check_logprobs(dev(np.where(r.random((M, V)) < .5, 0.0, -0.0)).half(), None, tok, 32)
    check_logprobs(dev(r.integers(0, 3, (M, V)).astype(np.float64)).bfloat16(), None, tok, 32)
    check_logprobs(dev(np.sort(r.integers(0, 50, (M, V)), axis=1).astype(np.float64)).half(), None, tok, 20)
    check_logprobs(dev(-np.sort(r.integers(0, 50, (M, V)), axis=1).astype(np.float64)).float(), None, tok, 20)


@pytest.mark.parametrize("M,V", [(1, 49152), (300, 49152), (2, 16000)])
@pytest.mark.parametrize("period", [512, 2048, 8192])
def test_logprobs_large_values_at_one_stride(M, V, period):
    """Rows whose large values all lie 8 in each `period`: one group of threads may hold them all."""
    r = rng(12, M, period)
    x = r.standard_normal((M, V)) * 0.1 - 5
    for first in (0, 3, 8 * 17):
        y = x.copy()
        at = np.arange(V)
        hit = (at - first) % period < 8
        y[:, hit] = r.standard_normal((M, hit.sum())) + 5
        check_logprobs(dev(y).half(), None, r.integers(0, V, M), 32)
        check_logprobs(dev(y).float(), None, r.integers(0, V, M), 20)


@pytest.mark.parametrize("V", [300, 49152, 200000])
def test_logprobs_masked_rows(V):
    r = rng(13, V)
    x = r.standard_normal((6, V))
    ninf = -np.inf
    x[0] = ninf                                    # nothing left
    x[1, 7:] = ninf                                # seven tokens left
    x[2, :] = ninf
    x[2, V - 1] = 1.5                              # one token left: certain
    x[3, V // 2] = np.nan
    x[4, 11] = np.inf
    X = dev(x).float()
    tok = dev(np.array([3, 100, V - 1, 5, 11, 9]))
    got = mnb.logprobs(X, tok, 20)
    lp, ent, tl, tt = (t.cpu().numpy() for t in got)
    assert np.isnan(lp[[0, 3, 4]]).all() and np.isnan(ent[[0, 3, 4]]).all() and np.isnan(tl[[0, 3, 4]]).all()
    assert tt[0].tolist() == list(range(20))       # all alike: the lowest indices
    assert tt[3, 0] == V // 2 and tt[4, 0] == 11   # NaN above all, infinity above numbers
    assert lp[1] == ninf and (tl[1, 7:] == ninf).all() and tt[1, 7:].tolist() == list(range(7, 20))
    live = ref.logprobs(f64(X)[1:2, :7], np.array([0]), 7)
    assert abs(ent[1] - live[1][0]) < 1e-5 and np.array_equal(tt[1, :7], live[4][0])
    assert lp[2] == 0 and ent[2] == 0 and tl[2, 0] == 0 and tt[2, 0] == V - 1
    check_logprobs(X[5:], None, np.array([9]), 20, mnb.LogProbs(got.logprob[5:], got.entropy[5:], got.top_logprobs[5:], got.top_tokens[5:]))


def test_logprobs_tokens_outside():
    x = dev(rng(14).standard_normal((4, 1000))).half()
    got = mnb.logprobs(x, dev(np.array([-1, -100, 1000, 1 << 40])), 2)
    lp = got.logprob.cpu().numpy()
    assert lp[0] == 0 and lp[1] == 0 and np.isnan(lp[2:]).all()
    only = mnb.logprobs(x)
    assert only.logprob is None and only.top_tokens is None and torch.equal(only.entropy, got.entropy)
    none = mnb.logprobs(x[:0], dev(np.zeros(0, np.int64)), 2)
    assert none.logprob.shape == (0,) and none.top_tokens.shape == (0, 2)


def test_logprobs_extreme_sizes_of_numbers():
    x = np.zeros((3, 5000))
    x[0] = -6e4
    x[0, 9] = 6e4                                  # all but one term vanish
    x[1] = np.linspace(-200, 200, 5000)
    x[2] = 6e4
    check_logprobs(dev(x).float(), None, np.array([9, 4999, 0]), 20)
    check_logprobs(dev(x).bfloat16(), None, np.array([9, 4999, 0]), 20)


# ------------------------------------------------------------------------------------------
# offsets past 32 bits, rows past one launch
# ------------------------------------------------------------------------------------------


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes and 2^31 elements: their last rows match the same rows alone."""
    M, V = 45000, 49152
    x = torch.zeros(M, V, dtype=torch.float16, device=DEV)
    x[-3:] = dev(rng(18).standard_normal((3, V))).half()
    tok = torch.arange(M, device=DEV)
    got = mnb.logprobs(x, tok, 5)
    check_logprobs(x[-3:].clone(), None, np.arange(M - 3, M), 5,
                   mnb.LogProbs(got.logprob[-3:], got.entropy[-3:], got.top_logprobs[-3:], got.top_tokens[-3:]))
    assert bool((got.top_tokens[0] == torch.arange(5, device=DEV)).all())
    w = torch.ones(V, dtype=torch.float16, device=DEV)
    for fmt in (FP4, FP8):
        q = mnb.mx_quantize(x, fmt)
        last = mnb.mx_quantize(x[-3:].clone(), fmt)
        assert torch.equal(q.codes[-3:], last.codes) and torch.equal(q.scales[-3:], last.scales)
        y = mnb.mx_dequantize(q)
        assert torch.equal(y[-3:], mnb.mx_dequantize(last)) and not bool(y[:-3].any())
        del q, y
    n = mnb.rmsnorm(x, w, residual=x)
    alone = mnb.rmsnorm(x[-3:].clone(), w, residual=x[-3:].clone())
    assert torch.equal(n.y[-3:], alone.y) and torch.equal(n.hidden[-3:], alone.hidden)


def test_product_offsets_past_32_bits():
    """Y of more than 2^32 bytes, and X rows that lie megabytes apart."""
    M, N, K = 45000, 49152, 64
    r = rng(19)
    (xq, xs), (wq, ws) = exact_operands(r, 64, N, K, FP8)
    w = mnb.mx_pack(to_mx(wq, ws, FP4))
    x64 = to_mx(xq, xs, FP8)
    want = mnb.mx_matmul(x64, w)
    rep = -(-M // 64)
    x = mnb.mx_tensor(x64.codes.repeat(rep, 1)[:M], x64.scales.repeat(rep, 1)[:M], FP8)
    y = mnb.mx_matmul(x, w)
    assert torch.equal(y[:64], want) and torch.equal(y[M // 64 * 64:], want[:M % 64])
    del y
    apart = torch.zeros(300, (1 << 23) - 16, dtype=torch.uint8, device=DEV)
    apart[:, :K] = x64.codes.repeat(5, 1)[:300]
    x2 = mnb.mx_tensor(apart[:, :K], x64.scales.repeat(5, 1)[:300], FP8)
    w2 = mnb.mx_pack(to_mx(wq[:200], ws[:200], FP4))
    assert torch.equal(mnb.mx_matmul(x2, w2), want[:, :200].repeat(5, 1)[:300])


def test_norm_rows_past_one_launch():
    x = dev(rng(20).standard_normal((1, 32))).half().repeat((1 << 20) + 5, 1)
    w = torch.ones(32, dtype=torch.float16, device=DEV)
    n = mnb.rmsnorm(x, w, residual=x, fmt=FP8, keep16=True)
    for t in (n.y, n.hidden, n.q.codes, n.q.scales):
        assert bool((t == t[:1]).all())


# ------------------------------------------------------------------------------------------
# together, on streams, in graphs
# ------------------------------------------------------------------------------------------


class Layer:
    """norm -> MX product -> norm -> 8-bit lm_head -> log probabilities, with the framework's own
    MatMulNBits as the head."""

    def __init__(self, seed, M, K=576, V=2000):
        r = rng(15, seed)
        self.x, self.res = dev(r.standard_normal((M, K))).half(), dev(r.standard_normal((M, K))).half()
        self.n1, self.n2 = dev(1 + .1 * r.standard_normal(K)).half(), dev(1 + .1 * r.standard_normal(K)).half()
        self.w = mnb.mx_quantize(dev(r.standard_normal((K, K)) * .05).half(), FP4)
        self.packed = mnb.mx_pack(self.w)
        self.codes = dev(r.integers(0, 256, (V, K), dtype=np.uint8))
        self.scales = dev(r.uniform(1e-4, 2e-3, (V, K // 32))).half()
        self.head = mnb.pack(self.codes, self.scales, None, 8)
        self.tok = dev(r.integers(0, V, M))
        self.ws = torch.zeros(mnb.mnb_workspace_bytes(M, V, K, 8, 0), dtype=torch.uint8, device=DEV)

    def run(self):
        a = mnb.rmsnorm(self.x, self.n1, residual=self.res, fmt=FP8)
        y = mnb.mx_matmul(a.q, self.packed)
        b = mnb.rmsnorm(y, self.n2, residual=a.hidden)
        logits = mnb.matmul(b.y, self.head, ws=self.ws)
        return a, y, b, logits, mnb.logprobs(logits, self.tok, 10)

    def check(self, got):
        """Each call against the 64-bit form of its own inputs."""
        a, y, b, logits, lp = got
        K = self.x.shape[1]
        want, h = ref.rmsnorm(f64(self.x), f64(self.res), f64(self.n1), 1e-6)
        check_mx(a.q, want, FP8, K)
        xv = ref.dequantize(a.q.codes.cpu().numpy(), a.q.scales.cpu().numpy(), FP8)
        wv = ref.dequantize(self.w.codes.cpu().numpy(), self.w.scales.cpu().numpy(), FP4)
        assert (np.abs(f64(y) - xv @ wv.T) <= product_bound(xv, wv, xv @ wv.T, K, torch.float16)).all()
        check16(b.y, ref.rmsnorm(f64(y), f64(a.hidden), f64(self.n2), 1e-6)[0], torch.float16, K)
        head = (f64(self.codes) - 128) * np.repeat(f64(self.scales), 32, 1)
        assert np.abs(f64(logits) - f64(b.y) @ head.T).max() < 2e-2
        check_logprobs(logits, None, self.tok.cpu().numpy(), 10, lp)


@pytest.mark.parametrize("M", [1, 8, 77])
def test_a_layer_and_its_head(M):
    layer = Layer(M, M)
    layer.check(layer.run())


def flat(v):
    if isinstance(v, torch.Tensor):
        return [v]
    if isinstance(v, mnb.MxTensor):
        return [v.codes, v.scales]
    return [t for x in v if x is not None for t in flat(x)]


@pytest.mark.parametrize("M", [1, 40])
def test_graph_replays_match_eager(M):
    layer = Layer(20 + M, M)
    layer.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        captured = layer.run()
    for rep in range(4):
        layer.x.copy_(dev(rng(16, rep).standard_normal(tuple(layer.x.shape))).half())
        g.replay()
        torch.cuda.synchronize()
        eager = layer.run()
        torch.cuda.synchronize()
        for a, b in zip(flat(captured), flat(eager)):
            assert torch.equal(a, b), rep


def test_two_streams_at_once():
    """The same calls on two streams, in flight together: neither disturbs the other."""
    layers = [Layer(30 + i, 24, V=20000) for i in range(2)]
    want = [flat(l.run()) for l in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(flat(layers[i].run()))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))
