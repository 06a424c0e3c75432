"""GPU results of the operators in include/mnb_decode.h against plain 64-bit references.

What the cache holds is compared bit for bit, tokens exactly; rounded outputs by half a step of their type and
the bounds derived beside each test.
"""
from __future__ import annotations

import numpy as np
import pytest

import _decode_ref as dref
from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def rng(*seed):
    return np.random.default_rng([20261209, *seed])


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


class Setup:
    """A cache with shuffled pages for sequences of given lengths; every byte of it 0xff (NaN scales) at first."""

    def __init__(self, r, lengths, hkv, D, S, width=None, spare=3, stride=0):
        self.lengths_host, self.hkv, self.D, self.S = list(lengths), hkv, D, S
        need = [-(-n // S) for n in lengths]
        self.width = width or max(1, max(need))
        count = sum(need) + spare
        order = list(r.permutation(count))
        self.pages_host = np.full((len(lengths), self.width), -7, np.int32)      # nothing may use the places behind a sequence
        for b, n in enumerate(need):
            for c in range(min(n, self.width)):
                self.pages_host[b, c] = order.pop()
        bytes_ = mnb.mnb_kv_page_bytes(hkv, D, S)
        data = torch.full((count, bytes_ + stride), 255, dtype=torch.uint8, device=DEV)
        self.cache = mnb.KvCache(data[:, :bytes_], hkv, D, S)
        self.data, self.pages, self.lengths = data, dev(self.pages_host), ints(lengths)

    def fill(self, k, v, dtype):
        """Whole sequences, one behind the other."""
        starts = np.concatenate([[0], np.cumsum(self.lengths_host)])
        if starts[-1]:
            mnb.kv_append(None, dev(k, dtype), dev(v, dtype), self.cache, self.pages, self.lengths, starts=ints(starts))
        return starts


def heads(r, n, h, D, dtype):
    x = r.standard_normal((n, h, D)) * np.exp(0.5 * r.standard_normal((h, D)))
    return torch.from_numpy(x).to(dtype)


# ------------------------------------------------------------------------------------------
# appending and reading back
# ------------------------------------------------------------------------------------------

APPEND = [  # lengths, starts or None, hq, hkv, D, page, rot, interleaved, norm
    ([1], None, 9, 3, 64, 16, 64, False, False),
    ([700, 1, 16, 17, 0, 333], None, 14, 2, 64, 32, 32, True, True),
    ([5], [0, 5], 1, 1, 128, 16, 128, False, True),
    ([40, 3, 0, 130], [0, 40, 41, 41, 90], 8, 2, 128, 64, 128, True, True),
    ([100, 2], [0, 64, 67], 4, 4, 96, 128, 48, False, True),       # a row before the second sequence's first token
    ([70], [0, 70], 20, 4, 96, 16, 96, True, False),
    ([33, 34], [0, 33, 67], 3, 1, 192, 16, 192, False, True),
    ([65], [0, 65], 8, 1, 256, 256, 256, False, True),
    ([19] * 130, None, 32, 8, 128, 16, 128, False, True),           # more sequences than a wave has lanes
    (list(range(1, 200)), [i for i in range(200)], 2, 2, 64, 16, 16, True, False),
    ([9], [0, 9], 0, 2, 128, 16, 0, False, False),
    ([1 << 16], [0, 3], 2, 1, 64, 65536, 64, False, True),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, dtype):
    lengths, starts, hq, hkv, D, S, rot, il, norm = APPEND[case]
    r, t = rng(1, case), DT[dtype]
    place = dref.places(lengths, starts)
    T = len(place)
    s = Setup(r, lengths, hkv, D, S, stride=64 if case % 2 else 0)
    before = s.data.clone()
    wide = heads(r, T, hq + 2 * hkv, D, t)                           # slices of one projection's output
    q, k, v = (wide[:, a:b] for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    on = wide.to(DEV)
    tab = mnb.rope_table(s.width * S, rot, device=DEV) if rot else None
    w = [heads(r, 1, 1, D, t)[0, 0] for _ in range(2)] if norm else [None, None]
    st = None if starts is None else ints(starts)
    got = mnb.kv_append(on[:, :hq] if hq else None, on[:, hq:hq + hkv], on[:, hq + hkv:], s.cache, s.pages, s.lengths, starts=st,
                        rope=tab, q_weight=None if w[0] is None else w[0].to(DEV), k_weight=None if w[1] is None else w[1].to(DEV),
                        interleaved=il)
    pos = np.array([p for _, p in place])
    there = pos >= 0
    rows = tab.cpu().numpy()[np.maximum(pos, 0)] if rot else None
    wn = [None if x is None else f64(x) for x in w]
    if hq:
        want = dref.norm_rotate(f64(q), wn[0], 1e-6, rows, il) * there[:, None, None]
        # half a step of the type, and the 32-bit products before it: at most 6 roundings of each of the two terms
        size = np.abs(dref.norm_rotate(np.abs(f64(q)), None if wn[0] is None else np.abs(wn[0]), 1e-6, None if rows is None else np.abs(rows) * np.where(
            np.arange(rot) < rot // 2, 1, -1), il))
        size = np.maximum(size, np.abs(want))
        assert (np.abs(f64(got) - want) <= np.abs(want) * torch.finfo(t).eps / 2 + 12 * 2.0 ** -24 * size + torch.finfo(t).smallest_normal * torch.finfo(t).eps).all()
    else:
        assert got is None
    kv, vv = mnb.kv_read(s.cache, s.pages, s.lengths, T, starts=st, dtype=torch.float32)
    kw = dref.fp4(dref.norm_rotate(f64(k), wn[1], 1e-6, rows, il))
    vw = dref.fp4(f64(v))
    assert np.array_equal(f64(kv), np.where(there[:, None, None], kw, 0)) and np.array_equal(f64(vv), np.where(there[:, None, None], vw, 0))
    # nothing but the rows' places was written
    written = torch.zeros_like(s.data, dtype=torch.bool)
    flat = written.as_strided((s.cache.pages, hkv, S * (D + D // 16)), (s.data.stride(0), S * (D + D // 16), 1))
    for b, p in place:
        if p < 0:
            continue
        h, i = flat[s.pages_host[b, p // S]], p % S
        h[:, i * D // 2:(i + 1) * D // 2] = True
        h[:, S * D + i * (D // 32):S * D + (i + 1) * (D // 32)] = True
        h[:, S * D // 2:S * D].view(hkv, S // 4, D // 8, 4, 4)[:, i // 4, :, i % 4] = True
        h[:, S * D + S * D // 32:].view(hkv, S // 4, D // 32, 4)[:, i // 4, :, i % 4] = True
    assert torch.equal(s.data[~written], before[~written])


def test_append_of_what_is_no_number():
    """Blocks of keys and values with NaN or infinities stand for NaN; a norm makes all of a key NaN."""
    r = rng(2)
    for norm in (False, True):
        s = Setup(r, [4], 2, 128, 16)
        k, v = heads(r, 4, 2, 128, torch.bfloat16), heads(r, 4, 2, 128, torch.bfloat16)
        k[1, 0, 40], v[2, 1, 100], k[3, 1, 0], v[0, 0, 5] = float("nan"), float("inf"), float("-inf"), 0.0
        v[3] = 0
        w = torch.ones(128, dtype=torch.bfloat16, device=DEV) if norm else None
        q = mnb.kv_append(k.to(DEV), k.to(DEV), v.to(DEV), s.cache, s.pages, s.lengths, starts=ints([0, 4]), q_weight=w, k_weight=w)
        kv, vv = mnb.kv_read(s.cache, s.pages, s.lengths, 4, starts=ints([0, 4]), dtype=torch.bfloat16)
        with np.errstate(invalid="ignore"):
            want = dref.norm_rotate(f64(k), 1.0 if norm else None, 1e-6, None, False)
        assert np.array_equal(f64(vv), dref.fp4(f64(v)), equal_nan=True)
        if norm:
            bad = np.zeros((4, 2), bool)
            bad[1, 0] = bad[3, 1] = True
            assert np.isnan(f64(kv)[1, 0]).all() and np.isnan(f64(kv)[3, 1, :32]).all() and np.isnan(f64(q)[1, 0]).all()
            assert np.array_equal(f64(kv)[~bad], dref.fp4(want)[~bad])
        else:
            assert np.array_equal(f64(kv), dref.fp4(f64(k)), equal_nan=True)


def test_rows_out_of_reach():
    """Pages out of range, positions past the pages or past the table: nothing stored, NaN; rows of no sequence untouched."""
    r = rng(3)
    s = Setup(r, [40, 40, 40, 70, 40], 2, 64, 16, width=4)
    s.pages[1, 2] = s.cache.pages                # the row at 39
    s.pages[2, 2] = -1
    tab = mnb.rope_table(39, 64, device=DEV)     # too short for position 39
    before = s.data.clone()
    x = heads(r, 8, 2, 64, torch.float16).to(DEV)
    out = torch.full((8, 2, 64), 7.0, dtype=torch.float16, device=DEV)
    starts = ints([0, 1, 2, 3, 4, 5])
    mnb.kv_append(x, x, x, s.cache, s.pages, s.lengths, starts=starts, rope=tab, out=out)
    assert torch.equal(s.data, before) and bool(out[:5].isnan().all()) and bool((out[5:] == 7).all())
    mnb.kv_append(x, x, x, s.cache, s.pages, s.lengths, starts=starts, out=out)
    assert not torch.equal(s.data, before) and not bool(out[[0, 4]].isnan().any()) and bool(out[1:4].isnan().all()) and bool((out[5:] == 7).all())
    kv = (torch.full_like(out, 7.0), torch.full_like(out, 7.0))
    mnb.kv_read(s.cache, s.pages, s.lengths, 8, starts=starts, out=kv)
    for t in kv:
        assert not bool(t[[0, 4]].isnan().any()) and bool(t[1:4].isnan().all()) and bool((t[5:] == 7).all())
    s.lengths.copy_(ints([40, 40, 40, 70, -5]))
    y = torch.full_like(out, 7.0)
    s.data.zero_()
    mnb.kv_attention(x, s.cache, s.pages, s.lengths, starts=starts, out=y)
    assert not bool(y[0].isnan().any()) and bool(y[1:4].isnan().all()) and bool((y[4] == 0).all()) and bool((y[5:] == 7).all())
    # far beyond: lengths of the largest number, starts that fall or pass the rows
    s.lengths.fill_(2 ** 31 - 1)
    mnb.kv_attention(x, s.cache, s.pages, s.lengths, starts=starts, out=y)
    mnb.kv_append(x, x, x, s.cache, s.pages, s.lengths, starts=starts, out=out)
    assert bool(y[:5].isnan().all()) and bool(out[:5].isnan().all())
    s.lengths.fill_(40)
    for bad in ([5, 3, 9, -1, 100, 2], [-5, 20, -5, 20, -5, 20], [2 ** 31 - 1, -2 ** 31, 0, 5, 3, 8]):
        mnb.kv_attention(x, s.cache, s.pages, s.lengths, starts=ints(bad), out=y)
        mnb.kv_append(x, x, x, s.cache, s.pages, s.lengths, starts=ints(bad), out=out)
        mnb.kv_read(s.cache, s.pages, s.lengths, 8, starts=ints(bad), out=kv)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------


def bound(y, size, t, score, n, D):
    """Half a step of the output; half a step for each probability in q's type (size is the sum of |p v|); of the scores, whose D
    products are summed in 32 bits and scaled (errors of (D + 4) steps of the largest |q k| sum, `score`, at most), twice
    the error, as it is in the numerator and in the sum; of the 32-bit sums over n tokens, of which a lane adds an eighth of a
    step of 32 at a time and the matrix instruction 32 at once, n / 4 + 64 roundings."""
    eps = torch.finfo(t).eps / 2
    return np.abs(y) * eps * 1.01 + size * (eps * 1.01 + 2 * (D + 4) * 2.0 ** -24 * score + (n / 4 + 64) * 2.0 ** -23) + 2.0 ** -24


ATTENTION = [  # lengths, starts or None, hq, hkv, D, page, window
    ([1], None, 1, 1, 64, 16, 0),
    ([1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65], None, 9, 3, 64, 16, 0),
    ([700, 129, 128, 127, 0], None, 14, 2, 64, 32, 0),
    ([255, 256, 257], None, 32, 8, 128, 64, 0),
    ([300, 40, 7], None, 20, 4, 96, 16, 50),
    ([513, 100], None, 3, 1, 192, 128, 0),
    ([400, 31, 0], None, 8, 1, 256, 16, 33),
    ([600], None, 40, 1, 128, 64, 0),                                 # more query heads than a tile has rows
    ([37], [0, 37], 4, 2, 128, 16, 0),                                # a prompt at once
    ([100, 50, 0, 3], [0, 5, 10, 10, 13], 9, 3, 64, 16, 0),           # a few rows each
    ([100, 2], [0, 7, 12], 4, 2, 96, 16, 20),                         # rows before the first token: zeros
    ([333, 200], [0, 100, 101], 14, 2, 64, 64, 100),
    ([90], [0, 45], 2, 2, 256, 32, 1),                                # each row sees itself alone
    ([150, 150, 150], [0, 33, 40, 100], 6, 2, 192, 16, 64),
]


def run_attention(r, lengths, starts, hq, hkv, D, S, window, t, scale=None, width=None, sharp=1.0):
    s = Setup(r, lengths, hkv, D, S, width=width)
    total, place = sum(lengths), dref.places(lengths, starts)
    k, v = heads(r, total, hkv, D, t), heads(r, total, hkv, D, t)
    at = s.fill(f64(k), f64(v), t)
    q = (heads(r, len(place), hq, D, t).double() * sharp).to(t)
    st = None if starts is None else ints(starts)
    y = mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths, starts=st, scale=scale, window=window)
    c = D ** -0.5 if scale is None else scale
    kq, vq, qf = dref.fp4(f64(k)), dref.fp4(f64(v)), f64(q)
    row = 0
    for b, n in enumerate(lengths):
        m = 1 if starts is None else starts[b + 1] - starts[b]
        kb, vb = kq[at[b]:at[b + 1]], vq[at[b]:at[b + 1]]
        want, size = dref.attention(qf[row:row + m], kb, vb, n - m, c, window)
        score = 0.0
        if m and n:
            score = float(np.max(np.einsum("nhd,thd->nht", np.abs(qf[row:row + m]), np.repeat(np.abs(kb), hq // hkv, 1)))) * abs(c)
        got = f64(y[row:row + m])
        err = np.abs(got - want)
        assert np.isfinite(got).all() and (err <= bound(want, size, t, score, n, D)).all(), (b, n, float(err.max()))
        row += m
    return s, q, y, st


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(case, dtype):
    run_attention(rng(4, case), *ATTENTION[case], DT[dtype])


@pytest.mark.parametrize("lengths,starts,hq,hkv,D,S,window", [
    ([5000], None, 14, 2, 64, 64, 0), ([3000, 10, 0, 900], None, 8, 2, 128, 16, 0), ([2100, 2100], [0, 3, 7], 10, 2, 96, 128, 0),
    ([4097], [0, 40], 4, 1, 128, 64, 0), ([3000, 3000], None, 4, 2, 256, 256, 2000), ([20000], None, 1, 1, 64, 65536, 0),
    ([1500] * 5 + [0] * 3, None, 2, 1, 192, 32, 0)])
def test_attention_split(lengths, starts, hq, hkv, D, S, window):
    """Sequences shared by several workgroups and joined."""
    r = rng(5, len(lengths), D)
    s, q, y, st = run_attention(r, lengths, starts, hq, hkv, D, S, window, torch.float16)
    c = mnb.mnb_kv_cache(None, 0, s.cache.pages, hkv, D, S)
    n = q.shape[0]
    rows = mnb.mnb_kv_rows(None, 0, None, 1 if starts else None, len(lengths), s.width, n)
    assert "join" in mnb.mnb_kv_describe_route(c, rows, hq, window)[1]
    again = mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths, starts=st, window=window)
    assert torch.equal(y, again)                                      # nothing depends on an order of arrival


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale,sharp", [(0.0, 1.0), (-0.3, 1.0), (2.0, 3.0), (1e-3, 1.0)])
def test_attention_scales(scale, sharp, dtype):
    """Flat, reversed and nearly one-hot distributions."""
    run_attention(rng(6), [200, 75], None, 4, 2, 128, 16, 0, DT[dtype], scale=scale, sharp=sharp)


def test_attention_far_apart_values():
    """bfloat16 keys and values far past what binary16 holds."""
    r, t = rng(7), torch.bfloat16
    lengths = [100]
    s = Setup(r, lengths, 2, 64, 16)
    k, v = heads(r, 100, 2, 64, t), heads(r, 100, 2, 64, t)
    k, v = (k.double() * 2.0 ** -40).to(t), (v.double() * torch.from_numpy(2.0 ** r.integers(-60, 60, (100, 1, 1)))).to(t)
    q = (heads(r, 1, 4, 64, t).double() * 2.0 ** 40).to(t)
    s.fill(f64(k), f64(v), t)
    y = mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths)
    want, size = dref.attention(f64(q), dref.fp4(f64(k)), dref.fp4(f64(v)), 99, 64 ** -0.5)
    assert (np.abs(f64(y) - want) <= bound(want, size, t, 60.0, 100, 64)).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_what_a_row_does_not_see(dtype, D):
    """NaN in keys and values of tokens behind a row, before its window and past the length does not reach it; of a token that it
    sees, a NaN block of values reaches these elements and no others, a NaN key all."""
    t, r, S, n, total = DT[dtype], rng(8, D), 16, 20, 70
    s = Setup(r, [total], 2, D, S)
    k, v = heads(r, total, 2, D, t), heads(r, total, 2, D, t)
    v[60, 0, D - 32], v[65, 1, 3], k[67, 0, 1], v[33, 0, 40] = float("nan"), float("inf"), float("nan"), float("nan")
    s.fill(f64(k), f64(v), t)
    q = heads(r, n, 6, D, t)
    y = f64(mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths, starts=ints([0, n]), window=21))
    want, size = dref.attention(f64(q), dref.fp4(f64(k)), dref.fp4(f64(v)), total - n, D ** -0.5, 21)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.isnan(want).any() and np.isfinite(want).any()
    ok = np.isfinite(want)
    assert (np.abs(y - want)[ok] <= bound(want, size, t, 8 * D ** 0.5, total, D)[ok]).all()


def test_views_and_in_place():
    """Rows inside wider ones, tables of pages inside wider ones, a cache of every second page, out in the place of q."""
    r, t = rng(9), torch.float16
    lengths, starts, hq, hkv, D, S = [90, 33], [0, 4, 9], 4, 2, 128, 16
    s = Setup(r, lengths, hkv, D, S)
    k, v = heads(r, 123, hkv, D, t), heads(r, 123, hkv, D, t)
    s.fill(f64(k), f64(v), t)
    q = heads(r, 9, hq, D, t).to(DEV)
    want = mnb.kv_attention(q, s.cache, s.pages, s.lengths, starts=ints(starts))
    wide = torch.full((9, hq + 3, D), 5.0, dtype=t, device=DEV)
    wide[:, 1:1 + hq] = q
    pages = torch.full((2, s.width + 5), -9, dtype=torch.int32, device=DEV)
    pages[:, 2:2 + s.width] = s.pages
    two = torch.zeros(2 * s.cache.pages, s.cache.data.shape[1], dtype=torch.uint8, device=DEV)
    two[1::2] = s.cache.data
    cache = mnb.KvCache(two[1::2], hkv, D, S)
    view, table = wide[:, 1:1 + hq], pages[:, 2:2 + s.width]
    got = mnb.kv_attention(view, cache, table, s.lengths, starts=ints(starts), out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(view, want)
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 1 + hq:] == 5).all()) and bool((two[::2] == 0).all())
    ver = wide._version
    args = (q[:, :2], cache, table, s.lengths, ints(starts), mnb.rope_table(96, 128, device=DEV))
    fresh = mnb.kv_append(view, wide[:, 5:], *args)
    assert wide._version == ver and mnb.kv_append(view, wide[:, 5:], *args, out=view) is not None
    assert wide._version == ver + 1 and torch.equal(view, fresh)
    with pytest.raises(RuntimeError, match="ALIAS"):
        mnb.kv_append(view, view[:, :2], *args, out=view)
    with pytest.raises(RuntimeError, match="ALIAS"):
        mnb.kv_attention(view, cache, table, s.lengths, starts=ints(starts), out=wide[:, 2:2 + hq])


def test_offsets_past_32_bits():
    """A cache of 5 GiB: pages beyond 2^32 bytes."""
    r, t, S, D, hkv = rng(10), torch.bfloat16, 65536, 128, 1
    bytes_ = mnb.mnb_kv_page_bytes(hkv, D, S)
    count = 5 * (1 << 30) // bytes_ + 1
    cache = mnb.kv_cache(count, hkv, D, page_size=S, device=DEV)
    pages, lengths = ints([count - 1, 0, count - 2, 5]).view(2, 2), ints([65600, 65536 + 17])
    n, starts = [200, 100], ints([0, 200, 300])
    k, v = heads(r, 300, hkv, D, t), heads(r, 300, hkv, D, t)
    # only the last rows are appended, and a window keeps the attention among them
    q = mnb.kv_append(k.to(DEV), k.to(DEV), v.to(DEV), cache, pages, lengths, starts=starts)
    kk, vv = mnb.kv_read(cache, pages, lengths, 300, starts=starts, dtype=t)
    assert np.array_equal(f64(kk), dref.fp4(f64(k))) and np.array_equal(f64(vv), dref.fp4(f64(v)))
    y = f64(mnb.kv_attention(q[[199, 299]], cache, pages, lengths, window=90))
    for i, (a, b) in enumerate(((0, 200), (200, 300))):
        want, size = dref.attention(f64(k[b - 1:b]), dref.fp4(f64(k[a:b])), dref.fp4(f64(v[a:b])), b - a - 1, D ** -0.5, 90)
        assert (np.abs(y[i:i + 1] - want) <= bound(want, size, t, 8 * D ** 0.5, 90, D)).all()


# ------------------------------------------------------------------------------------------
# sampling
# ------------------------------------------------------------------------------------------


def logits(r, M, V, dtype):
    x = r.standard_normal((M, V)) * 2
    x[np.arange(M)[:, None], r.integers(0, V, (M, min(8, V)))] += 4 + 3 * r.standard_normal((M, min(8, V)))
    return torch.from_numpy(x).to(dtype)


PARAMS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (0.9, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02), (2.5, 5, 0.3, 0.0),
          (0.0, 3, 0.5, 0.1), (1.0, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0), (0.05, 0, 0.999, 0.0), (30.0, 1000, 0.99, 1e-4),
          (1.0, 1 << 20, 2.0, -1.0), (1.0, -3, 1e-9, 7.0)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (5, 63), (40, 1000), (7, 4097), (3, 49152), (2, 50257), (2, 131072), (1, 262143)])
def test_sample(M, V, dtype):
    r = rng(11, M, V)
    x = logits(r, M, V, {"fp32": torch.float32, **DT}[dtype])
    xd, xf = x.to(DEV), f64(x)
    for t, k, p, m in PARAMS:
        u = r.random(M).astype(np.float32)
        u[0] = [0.0, 1.0 - 2.0 ** -24, 0.5][int(r.integers(3))]
        got = mnb.sample(xd, dev(u), t, k, p, m).cpu().numpy()
        t32, p32, m32 = np.float32(t), np.float32(p), np.float32(m)
        want = [dref.sample(xf[i], float(u[i]), float(t32), k, float(p32), float(m32)) for i in range(M)]
        assert got.tolist() == want, (t, k, p, m)
    # a row of its own parameters each
    pick = [PARAMS[i % len(PARAMS)] for i in range(M)]
    u = dev(r.random(M).astype(np.float32))
    cols = [torch.tensor([c[j] for c in pick], dtype=torch.int32 if j == 1 else torch.float32, device=DEV) for j in range(4)]
    each = mnb.sample(xd, u, *cols)
    for i in range(M):
        assert int(each[i]) == int(mnb.sample(xd[i:i + 1], u[i:i + 1], *pick[i])[0])


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_sample_ties_and_masks(dtype):
    """Rows of few distinct numbers, masked places at -infinity or the type's lowest value, both zeros."""
    t = {"fp32": torch.float32, **DT}[dtype]
    r, V = rng(12), 5000
    rows = [np.zeros(V), np.where(r.random(V) < 0.5, 0.0, -0.0), r.integers(0, 3, V).astype(float), np.where(r.random(V) < 0.999, -np.inf, 1.0),
            np.where(r.random(V) < 0.999, float(torch.finfo(t).min), r.standard_normal(V)), np.where(np.arange(V) == 4321, -3.0, -np.inf),
            np.full(V, float(torch.finfo(t).min)), np.full(V, float(torch.finfo(t).max)), np.repeat([5.0, 4.0, 3.0, -np.inf], V // 4)]
    x = torch.from_numpy(np.stack(rows)).to(t)
    xf = f64(x)
    for params in PARAMS:
        for u0 in (0.0, 0.1, 0.37, 0.5, 0.99, 1 - 2.0 ** -24):
            u = np.full(len(rows), u0, np.float32)
            got = mnb.sample(x.to(DEV), dev(u), *params).cpu().numpy().tolist()
            want = [dref.sample(xf[i], float(u[i]), *(float(np.float32(z)) if j != 1 else z for j, z in enumerate(params))) for i in range(len(rows))]
            assert got == want, (params, u0)


def test_sample_without_a_distribution():
    V = 300
    x = torch.randn(12, V, device=DEV)
    x[1, 7], x[2, 0], x[3], x[4, V - 1] = float("nan"), float("inf"), -float("inf"), float("nan")
    u = torch.full((12,), 0.5, device=DEV)
    t, p, m = torch.ones(12, device=DEV), torch.full((12,), 0.9, device=DEV), torch.zeros(12, device=DEV)
    u[5], t[6], t[7], t[8], p[9], m[10] = float("nan"), -1.0, float("nan"), float("inf"), float("nan"), float("nan")
    got = mnb.sample(x, u, t, 10, p, m).cpu().numpy()
    assert (got[1:11] == -1).all() and got[0] >= 0 and got[11] >= 0
    assert (mnb.sample(x, u, 0.0).cpu().numpy()[1:6] == -1).all()
    # u outside [0, 1) counts as the nearest number inside
    y = torch.randn(4, V, device=DEV)
    ends = mnb.sample(y, torch.tensor([-3.0, 0.0, 1.0, 5.0], device=DEV)).cpu().tolist()
    last = mnb.sample(y, torch.full((4,), 1 - 2.0 ** -24, device=DEV)).cpu().tolist()
    assert ends[:2] == [0, 0] and ends[2:] == last[2:]


def test_sample_views_and_repeats():
    r = rng(13)
    wide = logits(r, 6, 3000, torch.bfloat16).to(DEV)
    x = wide[:, 17:2018]
    u = torch.rand(6, device=DEV)
    want = mnb.sample(x.contiguous(), u, 0.9, 100, 0.97, 0.001)
    out = torch.empty(6, dtype=torch.int64, device=DEV)
    assert mnb.sample(x, u, 0.9, 100, 0.97, 0.001, out=out) is not None and torch.equal(out, want) and out._version == 1
    for _ in range(5):
        assert torch.equal(mnb.sample(x, u, 0.9, 100, 0.97, 0.001), want)


def test_sample_frequencies():
    """u on an even grid takes each token as often as its probability says, to one grid step for each border."""
    p = np.array([0.05, 0.3, 0.0, 0.15, 0.5])
    with np.errstate(divide="ignore"):
        x = torch.from_numpy(np.log(p)).float().to(DEV).expand(4000, 5).contiguous()
    u = ((torch.arange(4000, device=DEV).double() + 0.5) / 4000).float()
    got = np.bincount(mnb.sample(x, u).cpu().numpy(), minlength=5)
    assert (np.abs(got - 4000 * p) <= 1).all()


# ------------------------------------------------------------------------------------------
# attention of many rows (its reference in 64 bits on the GPU, by heads)
# ------------------------------------------------------------------------------------------


def attention64(q, k, v, first, scale, window):
    """dref.attention for [n, Hq, D] float64 tensors on the GPU: (y, sum of |p v|)."""
    n, hq, _ = q.shape
    p = first + torch.arange(n, device=DEV)[:, None]
    t = torch.arange(k.shape[0], device=DEV)[None]
    hidden = (t > p) | ((t <= p - window) if window else torch.zeros_like(t > p))
    blank = hidden.all(1)
    y, size = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(hq):
        kh, vh = (x[:, h // (hq // x.shape[1])].contiguous() for x in (k, v))
        s = (q[:, h].contiguous() @ kh.t().contiguous() * scale).masked_fill(hidden, -float("inf"))
        e = torch.softmax(s, 1).masked_fill(blank[:, None], 0.0)
        y[:, h], size[:, h] = e @ vh, e @ vh.abs()
    return y, size


def route(s, hq, rows, starts, window):
    c = mnb.mnb_kv_cache(None, 0, s.cache.pages, s.hkv, s.D, s.S)
    r = mnb.mnb_kv_rows(None, 0, None, 1 if starts else None, len(s.lengths_host), s.width, rows)
    return mnb.mnb_kv_describe_route(c, r, hq, window)[1]


MANY = [  # lengths, starts, hq, hkv, D, page, window
    ([1100, 300], [0, 1100, 1250], 64, 64, 64, 16, 0),
    ([700, 0, 650], [0, 700, 700, 1333], 52, 26, 96, 32, 100),
    ([2500], [0, 2111], 32, 8, 128, 64, 0),
    ([900, 1500, 40], [0, 333, 1600, 1640], 40, 40, 128, 128, 333),
    ([1000], [0, 1000], 36, 36, 192, 16, 0),
    ([1300, 129], [0, 777, 906], 40, 20, 256, 256, 0),
    ([500, 600], [0, 503, 1100], 56, 56, 128, 16, 0),             # rows before a sequence's first token
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_of_many_rows(case, dtype):
    lengths, starts, hq, hkv, D, S, window = MANY[case]
    t, r = DT[dtype], rng(20, case)
    s = Setup(r, lengths, hkv, D, S)
    total = sum(lengths)
    g = torch.Generator(device=DEV).manual_seed(case)
    k, v, q = (torch.randn(n, h, D, generator=g, device=DEV).mul(torch.exp(0.3 * torch.randn(h, D, generator=g, device=DEV))).to(t)
               for n, h in ((total, hkv), (total, hkv), (starts[-1], hq)))
    whole = [0, *np.cumsum(lengths).tolist()]
    mnb.kv_append(None, k, v, s.cache, s.pages, s.lengths, starts=ints(whole))
    assert route(s, hq, starts[-1], starts, window).startswith(f"kv_attention tile={32 if D <= 128 else 16}")
    out = torch.full_like(q, 7.0)
    y = mnb.kv_attention(q, s.cache, s.pages, s.lengths, starts=ints(starts), window=window, out=out)
    kq, vq = mnb.kv_read(s.cache, s.pages, s.lengths, total, starts=ints(whole), dtype=torch.float32)
    for b, n in enumerate(lengths):
        a, e = starts[b], starts[b + 1]
        if a == e:
            continue
        kb, vb = kq[whole[b]:whole[b + 1]].double(), vq[whole[b]:whole[b + 1]].double()
        want, size = attention64(q[a:e].double(), kb, vb, n - (e - a), D ** -0.5, window)
        score = float((q[a:e].double().abs().amax(0) * 1.0).amax() * kb.abs().amax()) * D ** 0.5
        err = (y[a:e].double() - want).abs()
        assert bool((err <= torch.from_numpy(bound(f64(want), f64(size), t, min(score, 60.0), n, D)).to(DEV)).all()), (b, float(err.max()))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_and_what_they_do_not_see(D):
    """NaN among later tokens, and in the bytes behind a sequence, reaches no earlier row."""
    n, H, S, t = 700, 96 if D < 256 else 48, 64, torch.bfloat16
    s = Setup(rng(21), [n], H, D, S)
    g = torch.Generator(device=DEV).manual_seed(D)
    q, k, v = (torch.randn(n, H, D, generator=g, device=DEV).to(t) for _ in range(3))
    v[600, 3, D - 1] = v[333, 0, 0] = float("nan")
    k[500, 2, 5] = float("inf")
    mnb.kv_append(None, k, v, s.cache, s.pages, s.lengths, starts=ints([0, n]))
    assert route(s, H, n, [0, n], 0).startswith(f"kv_attention tile={32 if D <= 128 else 16}")
    y = mnb.kv_attention(q, s.cache, s.pages, s.lengths, starts=ints([0, n]))
    bad = torch.zeros(n, H, D, dtype=torch.bool, device=DEV)
    bad[600:, 3, D - 32:] = bad[333:, 0, :32] = bad[500:, 2] = True
    assert torch.equal(y.isnan(), bad)


def test_many_rows_out_of_reach():
    """A page out of range, and more tokens than the pages hold: the rows of that sequence are NaN, others not; rows behind the
    last sequence stay."""
    n, H, D, S, t = 520, 44, 64, 64, torch.float16
    s = Setup(rng(22), [n, n, n + 200], H, D, S, width=9)
    s.data.zero_()
    s.pages[1, 4] = s.cache.pages
    q = torch.randn(3 * n + 5, H, D, device=DEV).to(t)
    out = torch.full_like(q, 7.0)
    starts = [0, n, 2 * n, 3 * n]
    assert route(s, H, 3 * n + 5, starts, 0).startswith("kv_attention tile=32")
    mnb.kv_attention(q, s.cache, s.pages, s.lengths, starts=ints(starts), out=out)
    assert not bool(out[:n].isnan().any()) and bool((out[3 * n:] == 7).all())
    assert bool(out[n + 64 * 4 + 128:2 * n].isnan().all()) and bool(out[2 * n:3 * n].isnan().all())
