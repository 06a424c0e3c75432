"""Which calls of attention may cut long items: by host sizes alone only those whose items cannot be long against the rounds of
them that a place on the card takes.  No GPU."""
from __future__ import annotations

import pytest

from _util import ensure_lib

mnb = ensure_lib()


def plan(batch, tokens, hq=32, hkv=8, D=128, S=64, rows=None, window=0):
    """(route, workspace bytes) of `batch` sequences in tables of `tokens` each, of one row or, together, `rows`."""
    width = -(-tokens // S)
    c = mnb.mnb_kv_cache(None, 0, 1, hkv, D, S)
    r = mnb.mnb_kv_rows(None, 0, None, None if rows is None else 1, batch, width, batch if rows is None else rows)
    st, text = mnb.mnb_kv_describe_route(c, r, hq, window)
    assert st == 0
    return text, mnb.mnb_kv_attention_workspace_bytes(c, r, hq, window)


@pytest.mark.parametrize("args", [
    dict(batch=1, tokens=131072), dict(batch=191, tokens=131072), dict(batch=192, tokens=131072), dict(batch=257, tokens=131072),
    dict(batch=4096, tokens=1 << 20), dict(batch=1 << 16, tokens=1 << 24), dict(batch=33, tokens=32768, rows=2080),
    dict(batch=65, tokens=16384, rows=2112), dict(batch=9, tokens=131072, rows=1032), dict(batch=512, tokens=16384, hq=14, hkv=2, D=64),
    dict(batch=600, tokens=65536, hq=8, hkv=8, D=256), dict(batch=257, tokens=131072, window=40000)])
def test_long_items_may_be_cut_in_any_batch(args):
    text, size = plan(**args)
    assert "join" in text and 0 < size < 1 << 25                 # the workspace is bounded by the card, not by the batch


@pytest.mark.parametrize("args", [
    dict(batch=1, tokens=1024), dict(batch=256, tokens=1024), dict(batch=256, tokens=2048), dict(batch=1, tokens=8192, rows=8192),
    dict(batch=1, tokens=2048, rows=2048), dict(batch=1, tokens=4096, hq=14, hkv=2, D=64, rows=4096), dict(batch=256, tokens=4096),
    dict(batch=1 << 16, tokens=32768), dict(batch=257, tokens=131072, window=1024)])
def test_items_that_cannot_be_long_take_one_launch(args):
    text, size = plan(**args)
    assert "join" not in text and size == 0
