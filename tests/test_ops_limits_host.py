"""The size limits of include/mnb_ops.h at their borders (host only)."""
from __future__ import annotations

import pytest

from _util import ensure_lib

mnb = ensure_lib()
pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_product_sizes():
    """ceil(M / 64) ceil(N / 128) <= 2^23 - 8, ceil(N / 64) ceil(K / 128) < 2^24, K < 2^22."""
    def route(M, N, K):
        return mnb.mnb_mx_describe_route(M, N, K, 1)[0]
    assert route(131072, 49152, 64) == OK and route(65536, 65536, 4096) == OK
    tiles = (1 << 23) - 8
    assert route(64 * tiles, 128, 32) == OK and route(64 * tiles + 1, 128, 32) == UNSUPPORTED
    assert route(1, 128 * tiles, 32) == OK and route(1, 128 * tiles + 1, 32) == UNSUPPORTED
    assert route(1, 64, (1 << 22) - 32) == OK and route(1, 64, 1 << 22) == UNSUPPORTED
    assert mnb.mnb_mx_packed_sizes(64 * ((1 << 24) - 1), 128)[0] == OK
    assert mnb.mnb_mx_packed_sizes(64 << 24, 128)[0] == UNSUPPORTED
    assert mnb.mnb_mx_packed_sizes(64 * ((1 << 23) - 1), 160)[0] == OK and mnb.mnb_mx_packed_sizes(64 << 23, 160)[0] == UNSUPPORTED


def test_logprobs_sizes():
    """Any number of rows (they go in several launches), V <= 2^22."""
    def ws(M, V, top=5):
        return mnb.mnb_logprobs_workspace_bytes(M, V, 0, top)
    far = 1 << 40
    assert ws(2000000, 262144) == 2000000 * 6 * (16 + 40) and ws(1 << 30, 8) == 0
    # a missing workspace is found after the sizes: nothing is refused for their product
    st = mnb.mnb_logprobs(far, 0, 2000000, 262144, 262144, 2 * far, 5, 3 * far, 4 * far, 5 * far, 6 * far, None, 0, None)
    assert st == 4
    assert mnb.mnb_logprobs(far, 0, 1, (1 << 22) + 1, 1 << 23, 2 * far, 0, 3 * far, 4 * far, None, None, None, 0, None) == UNSUPPORTED
