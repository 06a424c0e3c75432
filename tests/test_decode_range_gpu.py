"""Numbers at the ends of the ranges of include/mnb_decode.h, on the GPU, against plain 64-bit references."""
from __future__ import annotations

import numpy as np
import pytest

import _decode_ref as dref
from _util import ensure_lib
from test_decode_gpu import DEV, Setup, bound, dev, f64, heads, ints, rng

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("lengths,starts,hq,hkv,D,S,window", [
    ([200, 33, 1], None, 4, 2, 64, 16, 0), ([150, 70], [0, 5, 40], 6, 2, 96, 32, 60), ([3000], None, 8, 2, 128, 64, 0),
    ([100], [0, 100], 3, 1, 192, 16, 0), ([90, 64], [0, 40, 80], 4, 2, 256, 16, 0), ([1500], [0, 1500], 24, 24, 64, 64, 0)])
def test_keys_past_fp16(lengths, starts, hq, hkv, D, S, window, norm):
    """fp16 keys that a rotation (65504 turned by an eighth is 92637) or a weight takes past fp16 are in the cache as the numbers
    they are, and attention takes them so, among ordinary ones.  A key's blocks are exact in both parts of the product, which
    are summed in 32 bits as all scores are: the bound is theirs."""
    t, r = torch.float16, rng(30, len(lengths), D)
    s = Setup(r, lengths, hkv, D, S)
    total, place = sum(lengths), dref.places(lengths, starts)
    whole = [0, *np.cumsum(lengths).tolist()]
    k, v = heads(r, total, hkv, D, t), heads(r, total, hkv, D, t)
    large = torch.from_numpy(r.random((total, hkv, 1)) < 0.3) & (torch.arange(D) % (D // 2) < D // 4)      # both of a pair
    weight = None
    if norm:
        weight = torch.where(torch.arange(D) % 96 < 40, 60000.0, 1.0).to(t)
    else:
        k = torch.where(large, (60000 + 5000 * torch.from_numpy(r.random(k.shape))) * torch.sign(k.double()), k.double()).to(t)
    tab = mnb.rope_table(s.width * S, D, device=DEV)
    mnb.kv_append(None, k.to(DEV), v.to(DEV), s.cache, s.pages, s.lengths, starts=ints(whole), rope=tab,
                  k_weight=None if weight is None else weight.to(DEV))
    pos = np.concatenate([np.arange(n) for n in lengths])
    keys = dref.fp4(dref.norm_rotate(f64(k), None if weight is None else f64(weight), 1e-6, tab.cpu().numpy()[pos], False))
    values = dref.fp4(f64(v))
    assert (np.abs(keys) >= 65536).any() and np.isfinite(keys).all()
    q = (heads(r, len(place), hq, D, t).double() * 2.0 ** -14).to(t)
    c = D ** -0.5 * 0.25
    y = f64(mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths, starts=None if starts is None else ints(starts), scale=c, window=window))
    row = 0
    for b, n in enumerate(lengths):
        m = 1 if starts is None else starts[b + 1] - starts[b]
        kb, vb, qb = keys[whole[b]:whole[b + 1]], values[whole[b]:whole[b + 1]], f64(q[row:row + m])
        want, size = dref.attention(qb, kb, vb, n - m, c, window) if m <= 100 else (None, None)
        at = np.arange(m)
        if want is None:                                        # some rows are enough
            at = np.array([0, 1, 31, 32, m // 2, m - 1])
            got = [dref.attention(qb[i:i + 1], kb[:n - m + i + 1], vb[:n - m + i + 1], n - m + i, c, window) for i in at]
            want, size = (np.concatenate(x) for x in zip(*got))
        score = float(max(np.abs(qb[:, h] * 1.0).max(0) @ np.abs(kb[:, h // (hq // hkv)]).max(0) for h in range(hq))) * c
        assert np.isfinite(y[row:row + m]).all()
        assert (np.abs(y[row + at] - want) <= bound(want, size, t, score, n, D)).all(), (b, float(np.abs(y[row + at] - want).max()))
        row += m


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 96, 256])
def test_positions_past_the_table(D, t):
    """A row past the table is NaN, and so is what is read and attended to at its place, whatever the place held; nothing else is
    touched.  A row past the table and the pages stores nothing."""
    r, S, hkv, hq = rng(31, D), 16, 2, 4
    s = Setup(r, [40, 41, 20, 70], hkv, D, S, width=4)           # the last one lies past the pages
    s.data.zero_()
    old = heads(r, 101, hkv, D, t).to(DEV)
    old_starts = ints([0, 40, 81, 101, 101])
    mnb.kv_append(None, old, old, s.cache, s.pages, s.lengths, starts=old_starts)
    before = s.data.clone()
    x, q = heads(r, 4, hkv, D, t).to(DEV), heads(r, 4, hq, D, t).to(DEV)
    got = mnb.kv_append(q, x, x, s.cache, s.pages, s.lengths, rope=mnb.rope_table(39, 32, device=DEV))
    assert bool(got[[0, 1, 3]].isnan().all()) and bool(got[2].isfinite().all())
    k, v = mnb.kv_read(s.cache, s.pages, s.lengths, dtype=t)
    for y in (k, v):
        assert bool(y[[0, 1, 3]].isnan().all()) and bool(y[2].isfinite().all())
    # the scales of positions 39 and 40 are 255, and beside them only what the third row wrote has changed
    changed = (s.data != before).nonzero()
    places = {int(s.pages_host[0, 2]), int(s.pages_host[1, 2]), int(s.pages_host[2, 1])}
    assert set(changed[:, 0].tolist()) <= places
    for b, p in ((0, 39), (1, 40)):
        at = changed[changed[:, 0] == int(s.pages_host[b, 2])][:, 1].cpu().numpy() % (S * (D + D // 16))
        i = p % S
        mine = [*range(S * D + i * (D // 32), S * D + (i + 1) * (D // 32)),
                *(S * D + S * D // 32 + (i // 4 * (D // 32) + j) * 4 + i % 4 for j in range(D // 32))]
        assert sorted(set(at.tolist())) == sorted(mine)
    # whoever sees that place later gets NaN, with any query
    y = mnb.kv_attention(q, s.cache, s.pages, ints([40, 41, 20, 0]))
    assert bool(y[:2].isnan().all()) and bool(y[2].isfinite().all())
    y = mnb.kv_attention(q, s.cache, s.pages, ints([39, 40, 20, 0]))
    assert bool(y.isfinite().all())


# Sampling over a peak and a flat tail of tiny weights, which are whole numbers of 2^-S of the peak.  In such units a running
# sum rounds that of each eight neighbours once, V / 16 + 1; powers and exponents are off by 3 2^-52 of a weight, V / 22 of at most V
# weights of at most 2^46 units; u times the whole is rounded to 53 bits, V / 64; goal and running sum both have
# them: less than V / 4 + 4.
def unit(V):
    return 2.0 ** -min(46, 62 - int(np.ceil(np.log2(V))))


@pytest.mark.parametrize("tail", [-44.0, -41.2, -38.3, -30.0])
@pytest.mark.parametrize("V,peak", [(1 << 22, 1 << 21), ((1 << 22) - 5, (1 << 22) - 6), (131072, 70001)])
def test_sample_of_a_flat_tail(V, peak, tail):
    x = torch.full((1, V), tail * np.log(2.0), dtype=torch.float32, device=DEV)
    x[0, peak] = 0.0
    w = np.exp(f64(x)[0])
    end = np.cumsum(w)
    tol = (V / 4 + 4) * unit(V)
    r = rng(50, V, int(-tail))
    for u in [0.0, 1 - 2.0 ** -24, 0.5, *(r.random(6) * end[max(peak - 1, 0)] / end[-1])]:
        u = float(np.float32(u))
        got = int(mnb.sample(x, torch.tensor([u], device=DEV))[0])
        assert 0 <= got < V
        low, high, goal = (end[got - 1] if got else 0.0), end[got], u * end[-1]
        assert low - tol <= goal < high + tol, (u, got, peak)


@pytest.mark.parametrize("tail", [-38.3, -30.0, -24.5])
@pytest.mark.parametrize("V", [1 << 22, 131072])
def test_top_p_within_a_flat_tail(V, tail):
    """The border of top-p in the tail, seen by the last token that stays.  The sums that find it round each weight, and
    prefix and share of the whole are each off by V / 2 units for that, and by the other errors above: 5 V / 4; then those of u."""
    x = torch.full((1, V), tail * np.log(2.0), dtype=torch.float32, device=DEV)
    x[0, 0] = 0.0
    w = np.exp(f64(x)[0])
    end = np.cumsum(w)
    tol = (5 * V / 4 + V / 4 + 4) * unit(V)
    u = float(np.float32(1 - 2.0 ** -24))
    for share in (0.1, 0.5, 0.93):
        top_p = float(np.float32((1 + share * (end[-1] - 1)) / end[-1]))
        if top_p >= 1 or top_p * end[-1] <= 1:
            continue                                             # the tail is below a step of top_p
        got = int(mnb.sample(x, torch.tensor([u], device=DEV), 1.0, 0, top_p)[0])
        stays = min(V, int(np.searchsorted(end, top_p * end[-1])) + 1)
        want = u * end[stays - 1]
        assert end[got] > want - tol and (end[got - 1] if got else 0.0) < want + tol, (share, got, stays)
