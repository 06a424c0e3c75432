"""The operators of a decoding step as they are used: prompts and steps one behind the other, captured and replayed, on several
streams, and at the ends of their ranges.  Against 64-bit references; a replay against the eager call, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest

import _decode_ref as dref
from _util import ensure_lib
from test_decode_gpu import run_attention

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def bound(y, size, t, score, n, D):
    """Half a step of the output; of each probability half a step of q's type; twice the error of the scores (D products summed
    in 32 bits, (D + 4) steps of the largest sum of |q k|); and n / 4 + 64 roundings of the 32-bit sums over tokens."""
    eps = torch.finfo(t).eps / 2
    return np.abs(y) * eps * 1.01 + size * (eps * 1.01 + 2 * (D + 4) * 2.0 ** -24 * score + (n / 4 + 64) * 2.0 ** -23) + 2.0 ** -24


class Model:
    """One layer of attention between an embedding and a head over V tokens, for B sequences."""

    def __init__(self, seed, B, hq, hkv, D, V, S, most, t):
        g = torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.D, self.V, self.S, self.t = B, hq, hkv, D, V, S, t
        h = 96
        self.embed = torch.randn(V, h, generator=g).to(t).to(DEV)
        self.project = (torch.randn(h, (hq + 2 * hkv) * D, generator=g) * h ** -0.5).to(t).to(DEV)
        self.head = (torch.randn(hq * D, V, generator=g) * 0.3).to(t).to(DEV)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(t).to(DEV) for _ in range(2))
        self.table = mnb.rope_table(most, D // 2 // 16 * 16, device=DEV)
        width = -(-most // S)
        self.cache = mnb.kv_cache(B * width + 1, hkv, D, page_size=S, device=DEV)
        self.cache.data.fill_(255)
        self.pages = torch.randperm(B * width + 1, generator=g)[:B * width].view(B, width).int().to(DEV)

    def qkv(self, tokens):
        x = (self.embed[tokens] @ self.project).view(-1, self.hq + 2 * self.hkv, self.D)
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def rows(self, q, k, v, lengths, starts=None, window=0):
        q = mnb.kv_append(q, k, v, self.cache, self.pages, lengths, starts=starts, rope=self.table, q_weight=self.wq, k_weight=self.wk)
        return q, mnb.kv_attention(q, self.cache, self.pages, lengths, starts=starts, window=window)

    def logits(self, y):
        return y.reshape(y.shape[0], -1) @ self.head

    def step(self, tokens, lengths, u, window=0):
        _, y = self.rows(*self.qkv(tokens), lengths, window=window)
        return mnb.sample(self.logits(y), u, 0.8, 40, 0.95, 0.01)


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,D,S,window", [(9, 3, 64, 16, 0), (4, 1, 128, 32, 20), (6, 2, 96, 16, 0)])
def test_prompts_and_steps(hq, hkv, D, S, window, t):
    """Prompts of several lengths at once, then steps of a token each: attention against 64 bits on the keys that the 64-bit
    formula puts into the cache, tokens exactly those of the logits."""
    V, prompts, steps = 500, [1, 17, 40], 20
    m = Model(hq * D + window, len(prompts), hq, hkv, D, V, S, 80, t)
    tab, wq, wk = m.table.cpu().numpy(), f64(m.wq), f64(m.wk)
    r = np.random.default_rng(hq)
    keys, values = [[] for _ in prompts], [[] for _ in prompts]
    tokens = torch.from_numpy(r.integers(0, V, sum(prompts))).to(DEV)
    lengths, starts = list(prompts), [0, *np.cumsum(prompts).tolist()]
    for step in range(steps + 1):
        q, k, v = m.qkv(tokens)
        turned, y = m.rows(q, k, v, ints(lengths), None if starts is None else ints(starts), window)
        at = starts or list(range(len(prompts) + 1))
        for b, n in enumerate(lengths):
            rows = slice(at[b], at[b + 1])
            count = at[b + 1] - at[b]
            angle = tab[n - count:n]
            keys[b].append(dref.fp4(dref.norm_rotate(f64(k[rows]), wk, 1e-6, angle, False)))
            values[b].append(dref.fp4(f64(v[rows])))
            kb, vb = np.concatenate(keys[b]), np.concatenate(values[b])
            exact = dref.norm_rotate(f64(q[rows]), wq, 1e-6, angle, False)
            # half a step, and the 32-bit products before: at most 6 roundings of two terms no larger than the pair
            near = np.abs(exact).max(-1, keepdims=True) * 2 ** 0.5
            qf = f64(turned[rows])
            assert (np.abs(qf - exact) <= np.abs(exact) * torch.finfo(t).eps / 2 + 12 * 2.0 ** -24 * near + 2.0 ** -24).all()
            want, size = dref.attention(qf, kb, vb, n - count, D ** -0.5, window)
            score = float(np.einsum("nhd,thd->nht", np.abs(qf), np.repeat(np.abs(kb), hq // hkv, 1)).max()) * D ** -0.5
            assert (np.abs(f64(y[rows]) - want) <= bound(want, size, t, score, n, D)).all(), (step, b)
        last = torch.tensor([e - 1 for e in at[1:]], device=DEV)
        logits = m.logits(y[last])
        u = torch.from_numpy(r.random(len(prompts)).astype(np.float32)).to(DEV)
        tokens = mnb.sample(logits, u, 0.8, 40, 0.95, 0.01)
        x = f64(logits)
        assert tokens.tolist() == [dref.sample(x[b], float(u[b]), float(np.float32(0.8)), 40, float(np.float32(0.95)), float(np.float32(0.01)))
                                   for b in range(len(prompts))]
        lengths, starts = [n + 1 for n in lengths], None
    # the cache read back whole is what the formula put there
    lengths = [n - 1 for n in lengths]
    whole = [0, *np.cumsum(lengths).tolist()]
    kk, vv = mnb.kv_read(m.cache, m.pages, ints(lengths), whole[-1], starts=ints(whole), dtype=torch.float32)
    assert np.array_equal(f64(kk), np.concatenate([np.concatenate(x) for x in keys]))
    assert np.array_equal(f64(vv), np.concatenate([np.concatenate(x) for x in values]))


def test_captured_step():
    """A step of several hundred tokens' cache captured once, replayed as sequences grow, with eager work between."""
    t, B = torch.bfloat16, 3
    one, two = (Model(5, B, 8, 2, 128, 1000, 32, 2000, t) for _ in range(2))    # alike; one replays, the other runs eagerly
    start = [1200, 1, 640]
    fill = [0, *np.cumsum(start).tolist()]
    tokens = torch.from_numpy(np.random.default_rng(6).integers(0, 1000, fill[-1])).to(DEV)
    for m in (one, two):
        m.rows(*m.qkv(tokens), ints(start), ints(fill))
    now, lengths, u = tokens[:B].clone(), ints(start), torch.empty(B, device=DEV)
    def advance():
        lengths.add_(1)
        now.copy_(one.step(now, lengths, u))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    u.fill_(0.5)
    with torch.cuda.stream(side):                      # once before the capture, which the library calls among these need
        one.qkv(now), one.logits(torch.zeros(B, 8, 128, dtype=t, device=DEV))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        advance()
    token, n = now.clone(), lengths.clone()
    for i in range(12):
        u.copy_(torch.rand(B, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        n += 1
        token = two.step(token, n, u)
        assert torch.equal(token, now) and torch.equal(n, lengths)
        if i % 3 == 0:
            torch.cuda.synchronize()
        assert torch.equal(one.cache.data[one.pages[0].long()], two.cache.data[two.pages[0].long()])


def test_two_graphs_of_one_pool():
    """Two captured calls whose workspaces may share memory, replayed in turn and each several times."""
    t = torch.float16
    ms = [Model(7 + i, 2, 8, 2, 64, 64, 16, 9000, t) for i in range(2)]
    lengths = [ints([9000, 4000]), ints([300, 8111])]
    q = [torch.randn(2, 8, 64, device=DEV).to(t) for _ in ms]
    for m in ms:
        x = torch.randn(18000, 4, 64, device=DEV).to(t)
        mnb.kv_append(None, x[:, :2], x[:, 2:], m.cache, m.pages, ints([9000, 9000]), starts=ints([0, 9000, 18000]))
    want = [mnb.kv_attention(a, m.cache, m.pages, n) for a, m, n in zip(q, ms, lengths)]
    graphs, got = [torch.cuda.CUDAGraph() for _ in ms], []
    for i, (a, m, n) in enumerate(zip(q, ms, lengths)):
        with torch.cuda.graph(graphs[i], pool=graphs[0].pool() if i else None):
            got.append(mnb.kv_attention(a, m.cache, m.pages, n))
    for i in (0, 1, 1, 0, 0, 1):
        got[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(got[i], want[i])


def test_streams_at_once():
    """Calls of two streams under way together, each with its own workspace."""
    t = torch.bfloat16
    m = Model(11, 2, 16, 4, 128, 128, 64, 20000, t)
    x = torch.randn(40000, 8, 128, device=DEV).to(t)
    mnb.kv_append(None, x[:, :4], x[:, 4:], m.cache, m.pages, ints([20000, 20000]), starts=ints([0, 20000, 40000]))
    n = ints([20000, 12345])
    q = [torch.randn(2, 16, 128, device=DEV).to(t) for _ in range(2)]
    z = [torch.randn(8, 60000, device=DEV) for _ in range(2)]
    u = torch.rand(8, device=DEV)
    want = [(mnb.kv_attention(a, m.cache, m.pages, n), mnb.sample(b, u, 0.9, 0, 0.9)) for a, b in zip(q, z)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((mnb.kv_attention(q[i], m.cache, m.pages, n), mnb.sample(z[i], u, 0.9, 0, 0.9)))
    torch.cuda.synchronize()
    for i in range(2):
        for y, tokens in got[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(tokens, want[i][1])


@pytest.mark.parametrize("B", [63, 64, 65, 300])
def test_many_sequences(B):
    """More sequences than a wave has lanes, a third of them empty, whose rows are zeros; some of one row, some of several."""
    t, hq, hkv, D, S = torch.float16, 4, 2, 64, 16
    r = np.random.default_rng(B)
    lengths = np.where(r.random(B) < 0.33, 0, r.integers(1, 120, B))
    rows = np.where(lengths > 0, np.minimum(lengths, r.integers(0, 5, B)), 0)
    starts = np.concatenate([[0], np.cumsum(rows)])
    whole = np.concatenate([[0], np.cumsum(lengths)])
    cache = mnb.kv_cache(B * 8, hkv, D, page_size=S, device=DEV)
    cache.data.fill_(255)
    pages = torch.from_numpy(r.permutation(B * 8).reshape(B, 8).astype(np.int32)).to(DEV)
    k, v = (torch.from_numpy(r.standard_normal((whole[-1], hkv, D))).to(t) for _ in range(2))
    mnb.kv_append(None, k.to(DEV), v.to(DEV), cache, pages, ints(lengths), starts=ints(whole))
    kq, vq = dref.fp4(f64(k)), dref.fp4(f64(v))
    for st, first in ((starts, None), (None, 1)):
        n = B if st is None else int(starts[-1])
        q = torch.from_numpy(r.standard_normal((n, hq, D))).to(t)
        y = f64(mnb.kv_attention(q.to(DEV), cache, pages, ints(lengths), starts=None if st is None else ints(st)))
        at = np.arange(B + 1) if st is None else st
        for b in range(B):
            qb = f64(q[at[b]:at[b + 1]])
            if not lengths[b] or not len(qb):
                assert (y[at[b]:at[b + 1]] == 0).all()
                continue
            kb, vb = kq[whole[b]:whole[b + 1]], vq[whole[b]:whole[b + 1]]
            want, size = dref.attention(qb, kb, vb, int(lengths[b]) - len(qb), D ** -0.5, 0)
            score = float(np.einsum("nhd,thd->nht", np.abs(qb), np.repeat(np.abs(kb), hq // hkv, 1)).max()) * D ** -0.5
            assert (np.abs(y[at[b]:at[b + 1]] - want) <= bound(want, size, t, score, int(lengths[b]), D)).all(), b


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lengths,starts,hq,hkv,D,S,window", [
    ([4300, 10, 0, 900], None, 8, 2, 128, 16, 0), ([4200, 4100], [0, 3, 7], 10, 2, 96, 128, 0), ([4500, 4500], None, 4, 2, 256, 256, 4200),
    ([5000, 1500, 1500, 0], None, 2, 1, 192, 32, 0), ([6000, 300], [0, 70, 100], 8, 2, 128, 64, 0), ([1] * 70 + [6000], None, 4, 2, 64, 16, 0),
    ([200] * 40, None, 4, 2, 64, 2048, 0)])
def test_long_among_short(lengths, starts, hq, hkv, D, S, window, t):
    """Sequences long enough that an item is shared by workgroups whatever the others are, tiles of 32 rows too; and short ones in
    tables that could hold long ones, of which each item is one workgroup's."""
    _, q, y, st = run = run_attention(np.random.default_rng([len(lengths), D]), lengths, starts, hq, hkv, D, S, window, t)
    s = run[0]
    for _ in range(2):
        assert torch.equal(y, mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths, starts=st, window=window))


@pytest.mark.parametrize("hq,D,long", [(24, 128, 4200), (40, 64, 4200), (24, 96, 700)])
def test_many_heads_of_one(hq, D, long):
    """Tiles of 32 rows of a single token's heads: a short one, one and a part, an item shared by workgroups."""
    lengths = [long] + [150] * (39 if long > 1000 else 300)
    s, q, y, _ = run_attention(np.random.default_rng(D), lengths, None, hq, 1, D, 64, 0, torch.bfloat16)
    c = mnb.mnb_kv_cache(None, 0, s.cache.pages, 1, D, 64)
    text = mnb.mnb_kv_describe_route(c, mnb.mnb_kv_rows(None, 0, None, None, len(lengths), s.width, len(lengths)), hq, 0)[1]
    assert "tile=32" in text
    assert torch.equal(y, mnb.kv_attention(q.to(DEV), s.cache, s.pages, s.lengths))


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1 << 20, 1 << 22])
def test_sample_of_long_rows(V, t):
    """Rows up to the longest, top_k on both sides of what a workgroup sorts, and numbers that are equal thousands of times."""
    r = np.random.default_rng(V)
    x = torch.from_numpy(np.stack([r.standard_normal(V) * 3, np.round(r.standard_normal(V) * 4) / 4])).to(t)
    xd, xf = x.to(DEV), f64(x)
    for k, p, low in ((0, 1.0, 0.0), (150, 1.0, 0.0), (900, 0.9, 0.0), (5000, 1.0, 0.0), (100000, 0.7, 1e-3), (0, 0.3, 0.0)):
        u = r.random(2).astype(np.float32)
        got = mnb.sample(xd, torch.from_numpy(u).to(DEV), 0.9, k, p, low).tolist()
        want = [dref.sample(xf[i], float(u[i]), float(np.float32(0.9)), k, float(np.float32(p)), float(np.float32(low))) for i in range(2)]
        assert got == want, (k, p, low)


def test_inference_and_saved_tensors():
    """Outputs written in place count a version, tensors of inference mode have none."""
    m = Model(3, 1, 2, 1, 64, 32, 16, 32, torch.float16)
    q, k, v = (x.contiguous() for x in m.qkv(torch.tensor([5], device=DEV)))
    before = q._version
    mnb.kv_append(q, k, v, m.cache, m.pages, ints([1]), out=q)
    assert q._version == before + 1
    want = mnb.kv_attention(q, m.cache, m.pages, ints([1]))
    with torch.inference_mode():
        out = torch.empty_like(q)
        assert torch.equal(mnb.kv_attention(q, m.cache, m.pages, ints([1]), out=out), want)
        assert torch.equal(mnb.kv_attention(q.clone(), m.cache, m.pages, ints([1])), want)
