"""The calls with scratch and a second kernel (log probabilities of split rows) and the tiled product, in graphs that
are replayed between eager calls, in two graphs of one memory pool, and on two streams at once."""
from __future__ import annotations

import numpy as np
import pytest

from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")
FP4, FP8 = mnb.MNB_MX_FP4, mnb.MNB_MX_FP8


class Head:
    """norm -> MX product -> split-row log probabilities over V columns of a given type."""

    def __init__(self, seed, M, V, dtype=torch.float16, fmt=FP8, K=576):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, generator=g, device=DEV)
        assert mnb.mnb_logprobs_workspace_bytes(M, V, [torch.float16, torch.bfloat16, torch.float32].index(dtype), 20) > 0
        self.x, self.res, self.w = randn(M, K).half(), randn(M, K).half(), randn(K).half()
        self.packed = mnb.mx_pack(mnb.mx_quantize((randn(1000, K) * .05).half(), FP4))
        self.logits, self.fmt = (randn(M, V) * 3).to(dtype), fmt
        self.tok = torch.randint(0, V, (M,), generator=g, device=DEV)

    def new(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (self.x, self.res, self.logits):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))

    def run(self):
        n = mnb.rmsnorm(self.x, self.w, residual=self.res, fmt=self.fmt, keep16=True)
        y = mnb.mx_matmul(n.q, self.packed)
        return [n.y, n.hidden, n.q.codes, n.q.scales, y, *mnb.logprobs(self.logits, self.tok, 20)]

    def plain(self, got):
        """The scratch's results against 64 bits."""
        x = self.logits.double()
        logp = x - torch.logsumexp(x, 1, keepdim=True)
        size = 1 + np.log(x.shape[1])
        assert bool(((got[5].double() - logp.gather(1, self.tok[:, None])[:, 0]).abs() <= (logp.abs().amax() + size) * 2.0 ** -17).all())
        values, order = torch.sort(self.logits.float(), dim=1, descending=True, stable=True)
        assert torch.equal(got[8], order[:, :20])


def equal(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("M,V,dtype,fmt", [(1, 50257, torch.float16, FP8), (1, 131072, torch.float32, FP4), (40, 131072, torch.bfloat16, FP8),
                                           (300, 50257, torch.float16, FP4)])
def test_graph_replays(M, V, dtype, fmt):
    head = Head(1, M, V, dtype, fmt)
    head.plain(head.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        held = head.run()
    for rep in range(4):
        head.new(100 + rep)
        g.replay()
        torch.cuda.synchronize()
        eager = head.run()
        torch.cuda.synchronize()
        assert equal(held, eager), rep
        head.plain(held)


def test_two_graphs_of_one_pool():
    heads = [Head(2 + i, M, V) for i, (M, V) in enumerate(((3, 100000), (70, 65536)))]
    for h in heads:
        h.run()
    torch.cuda.synchronize()
    graphs, held, pool = [], [], None
    for h in heads:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            held.append(h.run())
        pool = g.pool()
        graphs.append(g)
    for rep in range(4):
        for i, h in enumerate(heads):
            h.new(200 + 10 * rep + i)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for h, got in zip(heads, held):
            assert equal(got, h.run()), rep
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 77])
def test_two_streams_at_once(M):
    heads = [Head(4 + i, M, 131072) for i in range(2)]
    want = [h.run() for h in heads]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in heads], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(heads[i].run())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(equal(run, want[i]) for run in got[i])
