"""What the calls of include/mnb_decode.h do with numbers that only the device sees and that are wrong: every buffer lies between
guards, and no byte but those of the call's own rows and pages changes."""
from __future__ import annotations

import numpy as np
import pytest

from _util import ensure_lib
from test_decode_gpu import DEV, ints, rng

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()

GUARD = 1 << 16                                       # bytes on either side
BAD_STARTS = [[5, 3, 9, -1, 100, 2], [-5, 20, -5, 20, -5, 20], [2 ** 31 - 1, -2 ** 31, 0, 5, 3, 8], [0, 8, 0, 8, 0, 8], [7, 7, 7, 7, 7, 7],
              [3, 4, 5, 6, 7, 2 ** 31 - 1], [0, 0, 0, 0, 0, 0]]


class Guarded:
    """A tensor of the given shape and type in the middle of a buffer of 0xa5."""

    def __init__(self, shape, dtype):
        self.bytes = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.whole = torch.full((2 * GUARD + self.bytes,), 0xa5, dtype=torch.uint8, device=DEV)
        self.t = self.whole[GUARD:GUARD + self.bytes].view(dtype).view(shape)

    def check(self, name):
        assert bool((self.whole[:GUARD] == 0xa5).all()) and bool((self.whole[GUARD + self.bytes:] == 0xa5).all()), name


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[40] * 5, [40, 0, 64, -7, 2 ** 31 - 1], [2 ** 31 - 1] * 5, [-2 ** 31, 64, 65, 1, 33]])
@pytest.mark.parametrize("D,S,hkv,hq", [(64, 16, 2, 2), (96, 32, 1, 4), (256, 16, 2, 4)])
def test_wrong_numbers_touch_nothing_else(D, S, hkv, hq, lengths, t):
    rows, batch, width = 8, 5, 64 // S
    need = mnb.mnb_kv_page_bytes(hkv, D, S)
    count = batch * width + 4
    pages = rng(40, D).permutation(count)[:batch * width].reshape(batch, width).astype(np.int32)
    free = sorted(set(range(count)) - set(pages.ravel().tolist()))
    pages[1, 0], pages[2, 1 % width], pages[4, width - 1] = count, -1, 2 ** 31 - 1
    data = Guarded((count, need + 64), torch.uint8)                   # 64 bytes behind each page belong to no one
    cache = mnb.KvCache(data.t[:, :need], hkv, D, S)
    q, y, kr, vr = (Guarded((rows, h, D), t) for h in (hq, hq, hkv, hkv))
    x = torch.randn(rows, hkv, D, device=DEV).to(t)
    tab = mnb.rope_table(50, 32, device=DEV)
    n = ints(lengths)
    p = torch.from_numpy(pages).to(DEV)
    inside = torch.zeros((count,), dtype=torch.bool, device=DEV)
    inside[[i for i in pages.ravel().tolist() if 0 <= i < count]] = True
    for bad in BAD_STARTS:
        st = ints(bad)
        start = data.t.clone()
        for rope in (None, tab):
            mnb.kv_append(torch.randn(rows, hq, D, device=DEV).to(t), x, x, cache, p, n, starts=st, rope=rope, out=q.t)
        assert torch.equal(data.t[:, need:], start[:, need:]) and torch.equal(data.t[free], start[free]) and torch.equal(data.t[~inside], start[~inside])
        held = data.t.clone()
        for window in (0, 7):
            mnb.kv_attention(q.t, cache, p, n, starts=st, window=window, out=y.t)
        mnb.kv_read(cache, p, n, rows, starts=st, dtype=t, out=(kr.t, vr.t))
        assert torch.equal(data.t, held)                             # reading changes nothing
        for g, name in ((data, "cache"), (q, "q"), (y, "y"), (kr, "k"), (vr, "v")):
            g.check((name, bad))
    torch.cuda.synchronize()


def test_wrong_numbers_where_work_is_shared():
    """The same for a call whose work is cut over workgroups and joined: workspace and results between guards, by the C call."""
    D, S, hkv, hq, rows, batch, width = 128, 16, 2, 8, 40, 5, 256
    need = mnb.mnb_kv_page_bytes(hkv, D, S)
    count = batch * width
    data = torch.zeros(count, need, dtype=torch.uint8, device=DEV)
    pages = torch.randperm(count, device=DEV).int().view(batch, width)
    cache = mnb.mnb_kv_cache(data.data_ptr(), need, count, hkv, D, S)
    q, y = torch.randn(rows, hq, D, device=DEV).half(), Guarded((rows, hq, D), torch.float16)
    for lengths in ([4096, 10, 0, 4000, 17], [2 ** 31 - 1, 4096, -3, 100, 4097]):
        n = ints(lengths)
        for bad in BAD_STARTS + [[0, 40, 1, 39, 2, 40], [0, 8, 16, 24, 32, 40]]:
            st = ints(bad)
            r = mnb.mnb_kv_rows(pages.data_ptr(), width, n.data_ptr(), st.data_ptr(), batch, width, rows)
            size = mnb.mnb_kv_attention_workspace_bytes(cache, r, hq, 0)
            assert size > 0 and "join" in mnb.mnb_kv_describe_route(cache, r, hq, 0)[1]
            ws = Guarded((size,), torch.uint8)
            st_ = mnb.mnb_kv_attention(cache, r, q.data_ptr(), hq * D, hq, 0, 0.1, 0, y.t.data_ptr(), hq * D, ws.t.data_ptr(), size,
                                       torch.cuda.current_stream().cuda_stream)
            assert st_ == 0
            y.check(("y", bad))
            ws.check(("workspace", bad))
            assert not bool(data.any())
    torch.cuda.synchronize()
