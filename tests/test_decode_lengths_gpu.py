"""Attention of large and mixed batches with a few sequences much longer than the others: their items are shared by workgroups while the
others' are taken whole.  Against the 64-bit reference, and bit for bit against itself."""
from __future__ import annotations

import numpy as np
import pytest

from _util import ensure_lib
from test_decode_gpu import DEV, DT, Setup, attention64, bound, f64, ints, rng, route, run_attention

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()


def again(s, q, y, st, window):
    out = torch.full_like(y, 7.0)
    for _ in range(3):
        assert torch.equal(y, mnb.kv_attention(q.to(y.device), s.cache, s.pages, s.lengths, starts=st, window=window, out=out))
        out.fill_(7.0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("where", ["first", "last", "both", "inside", "none"])
def test_one_row_each(where, dtype):
    """1600 items, of which those of the long sequences are cut (none: items of more than the least that is cut, none longer than an even share)."""
    r = rng(60)
    lengths = [int(x) for x in r.integers(0, 90, 100)]
    for i in dict(first=[0], last=[99], both=[0, 99], inside=[37, 70], none=[])[where]:
        lengths[i] = 9001 if i != 70 else 6000
    s, q, y, st = run_attention(r, lengths, None, 16, 16, 64, 16, 0, DT[dtype], width=600)
    assert "join" in route(s, 16, 100, None, 0)
    again(s, q, y, st, 0)


def test_all_long_and_alike():
    """Items long enough to be cut that are not, as none is longer than an even share: the workgroups that could share them
    leave all as it is.  (The reference in 64 bits on the GPU, of what the cache gives back.)"""
    r = rng(61)
    B, H, D, t = 100, 16, 64, torch.bfloat16
    lengths = [5300 + int(x) for x in r.integers(0, 50, B)]
    s = Setup(r, lengths, H, D, 64, width=96)
    whole = ints([0, *np.cumsum(lengths).tolist()])
    g = torch.Generator(device=DEV).manual_seed(61)
    k, v = (torch.randn(sum(lengths), H, D, generator=g, device=DEV).to(t) for _ in range(2))
    q = torch.randn(B, H, D, generator=g, device=DEV).to(t)
    mnb.kv_append(None, k, v, s.cache, s.pages, s.lengths, starts=whole)
    kq, vq = mnb.kv_read(s.cache, s.pages, s.lengths, sum(lengths), starts=whole, dtype=torch.float32)
    y = mnb.kv_attention(q, s.cache, s.pages, s.lengths)
    assert "join" in route(s, H, B, None, 0)
    at = 0
    for b, n in enumerate(lengths):
        want, size = attention64(q[b:b + 1].double(), kq[at:at + n].double(), vq[at:at + n].double(), n - 1, D ** -0.5, 0)
        # normal numbers: the largest sum of 64 |q k| over 8 lies below 30
        assert (np.abs(f64(y[b:b + 1]) - f64(want)) <= bound(f64(want), f64(size), t, 30.0, n, D)).all(), b
        at += n
    again(s, q, y, None, 0)


@pytest.mark.parametrize("hq,hkv,D,S,window,tile", [(64, 32, 64, 64, 0, 16), (96, 32, 64, 64, 0, 32), (32, 32, 128, 16, 0, 16), (32, 32, 96, 32, 8000, 16), (16, 16, 256, 64, 0, 16),
                                                    (40, 20, 192, 128, 0, 16)])
def test_a_prompts_part_beside_long_ones(hq, hkv, D, S, window, tile):
    """Rows of a prompt's part, several rows, single rows, sequences without rows or tokens, and rows before a sequence's first token, in one
    call with sequences of thousands of tokens."""
    r = rng(62, D)
    rows = [300, 1, 0, 1, 5, 1, 1, 3] + [1] * 40
    lengths = [400, 9000, 900, 12, 60, 3100, 0, 2] + [int(x) for x in r.integers(1, 60, 38)] + [8193, 7]
    starts = [0, *np.cumsum(rows).tolist()]
    s, q, y, st = run_attention(r, lengths, starts, hq, hkv, D, S, window, torch.float16)
    text = route(s, hq, starts[-1], starts, window)
    assert "join" in text and f"tile={tile}" in text
    again(s, q, y, st, window)


def test_captured_while_lengths_grow():
    """One captured call whose lengths change between replays, from no long sequence to one, two and none again."""
    r = rng(63)
    full = [9000] + [80] * 98 + [7000]
    s, q, y, st = run_attention(r, full, None, 16, 16, 64, 16, 0, torch.float16)
    qd = q.to(y.device)
    graph, n = torch.cuda.CUDAGraph(), s.lengths.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = mnb.kv_attention(qd, s.cache, s.pages, n)
    for lengths in (full, [50] + [80] * 99, [9000] + [1] * 99, [80] * 99 + [7000], [0] * 100, full):
        n.copy_(ints(lengths))
        got.fill_(7.0)
        graph.replay()
        want = mnb.kv_attention(qd, s.cache, s.pages, ints(lengths))
        torch.cuda.synchronize()
        assert torch.equal(got, want) and bool(got.isfinite().all())
    assert torch.equal(got, y)
