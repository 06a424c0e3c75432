"""Host-side checks of include/mnb_decode.h that need no GPU: exported names, sizes, routes, argument validation
before any device call, the torch binding's refusals, and the references that the GPU tests compare with."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

import _decode_ref as dref
from _util import ROOT, ensure_lib

mnb = ensure_lib()
torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, ALIAS = 0, 1, 2, 3, 4, 5
P = [(i + 1) << 40 for i in range(16)]     # far apart, never dereferenced


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mnb_decode.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mnb_[a-z_]+)\s*\(", text)))
    assert len(names) == 8
    for n in names:
        assert hasattr(mnb.lib, n) and callable(getattr(mnb, n)), n
    assert mnb.mnb_decode_version() == 100


def test_the_structs_are_those_of_the_header():
    assert ctypes.sizeof(mnb.mnb_kv_cache) == 32 and ctypes.sizeof(mnb.mnb_kv_rows) == 48
    assert mnb.mnb_kv_cache.page_size.offset == 28 and mnb.mnb_kv_rows.rows.offset == 40


def cache(data=P[0], stride=None, pages=10, heads=2, D=128, S=64):
    return mnb.mnb_kv_cache(data, heads * S * (D + D // 16) if stride is None else stride, pages, heads, D, S)


def rows(pages=P[1], ldp=8, lengths=P[2], starts=None, batch=4, width=8, n=None):
    return mnb.mnb_kv_rows(pages, ldp, lengths, starts, batch, width, batch if n is None else n)


def test_page_bytes():
    assert mnb.mnb_kv_page_bytes(8, 128, 64) == 8 * 64 * 136 and mnb.mnb_kv_page_bytes(3, 64, 16) == 3 * 16 * 68
    for heads, D, S in ((1, 80, 64), (1, 0, 64), (1, 128, 8), (1, 128, 48), (1, 128, 1 << 17), (-1, 128, 64), (1 << 20, 128, 64)):
        assert mnb.mnb_kv_page_bytes(heads, D, S) == 0


def append(c=None, r=None, q=P[3], ldq=1024, hq=8, k=P[4], ldk=256, v=P[5], ldv=256, dt=0, tab=P[6], tr=512, rot=128, il=0, qw=P[7],
           kw=P[8], eps=1e-6, out=P[9], ldo=1024):
    return mnb.mnb_kv_append(c or cache(), r or rows(), q, ldq, hq, k, ldk, v, ldv, dt, tab, tr, rot, il, qw, kw, eps, out, ldo, None)


COMMON = [(dict(c=cache(D=80)), UNSUPPORTED), (dict(c=cache(S=48)), UNSUPPORTED), (dict(c=cache(pages=-1)), INVALID),
          (dict(c=cache(stride=16)), INVALID), (dict(c=cache(data=P[0] + 8)), MISALIGNED), (dict(c=cache(data=None)), INVALID),
          (dict(c=cache(stride=2 * 64 * 136 + 8)), MISALIGNED), (dict(c=cache(pages=0)), INVALID),
          (dict(r=rows(n=5)), INVALID), (dict(r=rows(batch=-1, n=4)), INVALID), (dict(r=rows(lengths=None)), INVALID),
          (dict(r=rows(ldp=7)), INVALID), (dict(r=rows(pages=P[1] + 2)), MISALIGNED), (dict(r=rows(pages=None)), INVALID),
          (dict(r=rows(width=1 << 25, ldp=1 << 25)), UNSUPPORTED), (dict(r=rows(starts=P[10], n=1 << 22)), UNSUPPORTED),
          (dict(r=rows(starts=P[10] + 1)), MISALIGNED)]


@pytest.mark.parametrize("args,want", COMMON + [
    (dict(dt=2), INVALID), (dict(hq=-1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(tab=None), INVALID), (dict(rot=144), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(tr=-1), INVALID),
    (dict(ldq=1016), INVALID), (dict(ldk=128), INVALID), (dict(ldo=100), INVALID), (dict(ldq=1028), MISALIGNED), (dict(k=P[4] + 2), MISALIGNED),
    (dict(qw=P[7] + 2), MISALIGNED), (dict(tab=P[6] + 4), MISALIGNED),
    (dict(out=P[3] + 16), ALIAS), (dict(out=P[4]), ALIAS), (dict(out=P[0] + 4096), ALIAS), (dict(k=P[0]), ALIAS), (dict(out=P[2]), ALIAS),
    (dict(r=rows(pages=P[0])), ALIAS), (dict(r=rows(lengths=P[0] + 16)), ALIAS), (dict(tab=P[0]), ALIAS), (dict(kw=P[0] + 64), ALIAS),
    (dict(out=P[3], ldo=2048), ALIAS),
    (dict(r=rows(batch=0), q=None, k=None), INVALID), (dict(r=rows(batch=0), k=None), OK), (dict(r=rows(starts=P[10], n=0)), OK)])
def test_append_validation(args, want):
    assert append(**args) == want


def read(c=None, r=None, k=P[4], ldk=256, v=P[5], ldv=256, dt=0):
    return mnb.mnb_kv_read(c or cache(), r or rows(), k, ldk, v, ldv, dt, None)


@pytest.mark.parametrize("args,want", COMMON + [
    (dict(dt=3), INVALID), (dict(k=None, v=None), OK), (dict(ldk=255), INVALID), (dict(ldv=260), MISALIGNED), (dict(dt=2, ldv=258), MISALIGNED),
    (dict(k=P[5]), ALIAS), (dict(k=P[0]), ALIAS), (dict(v=P[1]), ALIAS)])
def test_read_validation(args, want):
    assert read(**args) == want


def attention(c=None, r=None, q=P[3], ldq=1024, hq=8, dt=0, scale=0.1, window=0, y=P[4], ldy=1024, ws=P[5], wsb=1 << 30):
    return mnb.mnb_kv_attention(c or cache(), r or rows(), q, ldq, hq, dt, scale, window, y, ldy, ws, wsb, None)


@pytest.mark.parametrize("args,want", COMMON + [
    (dict(dt=2), INVALID), (dict(hq=7), INVALID), (dict(hq=-2), INVALID), (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(y=None), INVALID), (dict(ldq=1023), INVALID), (dict(ldy=1028), MISALIGNED),
    (dict(y=P[3] + 16), ALIAS), (dict(y=P[0] + 64), ALIAS), (dict(y=P[2]), ALIAS), (dict(y=P[3], ldy=2048), ALIAS),
    (dict(r=rows(width=512, ldp=512), ws=None, wsb=0), WORKSPACE), (dict(r=rows(width=512, ldp=512), ws=P[5] + 8), MISALIGNED),
    (dict(r=rows(width=512, ldp=512), ws=P[3]), ALIAS), (dict(r=rows(width=512, ldp=512), ws=P[0]), ALIAS),
    (dict(hq=0, q=None), OK), (dict(r=rows(batch=0), q=None), OK), (dict(c=cache(heads=0), q=None), OK)])
def test_attention_validation(args, want):
    assert attention(**args) == want


def test_attention_workspace_and_route():
    def ws(r, c=None, hq=8, window=0):
        return mnb.mnb_kv_attention_workspace_bytes(c or cache(), r, hq, window)

    def route(r, c=None, hq=8, window=0):
        st, text = mnb.mnb_kv_describe_route(c or cache(), r, hq, window)
        assert st == OK
        return text
    assert ws(rows(width=2)) == 0 and "join" not in route(rows(width=2))
    long = rows(width=2048, ldp=2048)
    need = ws(long)
    assert need > 0 and "join" in route(long)
    assert attention(r=long, wsb=need - 1) == WORKSPACE
    assert ws(long, window=100) == 0                           # a short window leaves little to split
    assert ws(long, window=1 << 30) == need and ws(long, hq=7) == 0
    assert route(rows(batch=0)) == "noop"
    assert mnb.mnb_kv_describe_route(cache(), long, 7, 0)[0] == INVALID


def sample(x=P[0], dt=0, M=4, V=100, ldl=100, u=P[1], t=None, ta=1.0, k=None, ka=0, p=None, pa=1.0, m=None, ma=0.0, out=P[2]):
    return mnb.mnb_sample(x, dt, M, V, ldl, u, t, ta, k, ka, p, pa, m, ma, out, None)


@pytest.mark.parametrize("args,want", [
    (dict(M=0, x=None), OK), (dict(M=-1), INVALID), (dict(V=-1), INVALID), (dict(V=0), INVALID), (dict(dt=3), INVALID),
    (dict(V=(1 << 22) + 1, ldl=1 << 23), UNSUPPORTED), (dict(x=None), INVALID), (dict(u=None), INVALID), (dict(out=None), INVALID),
    (dict(ldl=99), INVALID), (dict(x=P[0] + 1), MISALIGNED), (dict(x=P[0] + 2, dt=2), MISALIGNED), (dict(u=P[1] + 2), MISALIGNED),
    (dict(out=P[2] + 4), MISALIGNED), (dict(t=P[3] + 1), MISALIGNED), (dict(k=P[3] + 2), MISALIGNED),
    (dict(out=P[0] + 8), ALIAS), (dict(out=P[1]), ALIAS), (dict(t=P[2]), ALIAS), (dict(k=P[2] + 8), ALIAS)])
def test_sample_validation(args, want):
    assert sample(**args) == want


# ------------------------------------------------------------------------------------------
# the torch binding's own checks (CPU tensors; every case fails before any library call)
# ------------------------------------------------------------------------------------------


def host_cache(pages=4, heads=2, D=64, S=16):
    return mnb.kv_cache(pages, heads, D, page_size=S, device="cpu")


def test_cache_refusals():
    for args in ((4, 2, 80, 16), (4, 2, 64, 24), (4, 0, 64, 16)):
        with pytest.raises(ValueError):
            mnb.kv_cache(*args[:3], page_size=args[3], device="cpu")
    need = mnb.mnb_kv_page_bytes(2, 64, 16)
    wide = torch.zeros(4, need + 32, dtype=torch.uint8)
    assert mnb.KvCache(wide[:, :need], 2, 64, 16).pages == 4
    with pytest.raises(TypeError):
        mnb.KvCache(wide.int(), 2, 64, 16)
    for bad in (wide[:, :need - 16], wide[:, 8:], torch.zeros(4, need + 8, dtype=torch.uint8), wide[0], wide.t()):
        with pytest.raises(ValueError):
            mnb.KvCache(bad, 2, 64, 16)


def heads(n, h, D=64, dtype=torch.float16):
    return torch.zeros(n, h, D, dtype=dtype)


def test_append_refusals():
    c, q, k, v = host_cache(), heads(3, 4), heads(3, 2), heads(3, 2)
    pages, lengths, starts = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    w, tab = torch.ones(64, dtype=torch.float16), mnb.rope_table(32, 64, device="cpu")

    def refused(kind, match="", **more):
        a = dict(q=q, k=k, v=v, cache=c, pages=pages, lengths=lengths, **{})
        a.update(more)
        with pytest.raises(kind, match=match):
            mnb.kv_append(**a)
    refused(ValueError, "on a GPU")
    refused(ValueError, "on a GPU", starts=starts, rope=tab, q_weight=w, k_weight=w, out=q)
    refused(TypeError, "tensor", k=3)
    refused(TypeError, "tensor", q=3)
    refused(TypeError, "tensor", pages=[[0]])
    refused(TypeError, "float16", k=k.float())
    refused(TypeError, "v must", v=v.bfloat16())
    refused(ValueError, "shape", k=k[:, :1])
    refused(ValueError, "shape", k=k[..., :32])
    refused(ValueError, "shape", q=q[:2])
    refused(ValueError, "side by side", q=torch.zeros(3, 4, 128, dtype=torch.float16)[..., :64])
    refused(ValueError, "overlap", v=v[:1].expand(3, 2, 64))
    refused(TypeError, "int32", pages=pages.long())
    refused(TypeError, "lengths", lengths=lengths.long())
    refused(ValueError, "lengths", lengths=lengths[:2])
    refused(ValueError, "starts", starts=starts[:3])
    refused(ValueError, "one row", q=q[:2], k=k[:2], v=v[:2])
    refused(ValueError, "contiguous", pages=pages.t().contiguous().t())
    refused(TypeError, "rope", rope=tab.half())
    refused(ValueError, "rope", rope=tab[:, :40])
    refused(ValueError, "rope", rope=torch.zeros(32, 24))
    refused(ValueError, "rope", rope=torch.zeros(32, 80))
    refused(TypeError, "q_weight", q_weight=w.float())
    refused(ValueError, "k_weight", k_weight=w[:32])
    refused(ValueError, "out needs q", q=None, out=q)
    refused(ValueError, "shape", out=q[:, :2])
    refused(TypeError, "out", out=q.float())
    refused(TypeError, "", eps="x")


def test_read_attention_and_sample_refusals():
    c, q = host_cache(), heads(3, 4)
    pages, lengths, starts = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.arange(4, dtype=torch.int32)
    for kind, match, call in (
            (ValueError, "on a GPU", lambda: mnb.kv_read(c, pages, lengths)),
            (ValueError, "rows is needed", lambda: mnb.kv_read(c, pages, lengths, starts=starts)),
            (ValueError, "one row", lambda: mnb.kv_read(c, pages, lengths, 2)),
            (ValueError, "negative", lambda: mnb.kv_read(c, pages, lengths, -1, starts=starts)),
            (TypeError, "output", lambda: mnb.kv_read(c, pages, lengths, dtype=torch.float64)),
            (ValueError, "shape", lambda: mnb.kv_read(c, pages, lengths, out=(heads(3, 1), None))),
            (ValueError, "on a GPU", lambda: mnb.kv_attention(q, c, pages, lengths, starts, 0.5, 7)),
            (TypeError, "float16", lambda: mnb.kv_attention(q.float(), c, pages, lengths)),
            (ValueError, "multiple", lambda: mnb.kv_attention(q[:, :3], c, pages, lengths)),
            (ValueError, "one row", lambda: mnb.kv_attention(q[:2], c, pages, lengths)),
            (ValueError, "window", lambda: mnb.kv_attention(q, c, pages, lengths, window=-1)),
            (ValueError, "shape", lambda: mnb.kv_attention(q, c, pages, lengths, out=q[:, :2])),
            (TypeError, "", lambda: mnb.kv_attention(q, c, pages, lengths, scale="x")),
            (ValueError, "side by side", lambda: mnb.kv_attention(q.transpose(0, 1).contiguous().transpose(0, 1), c, pages, lengths))):
        with pytest.raises(kind, match=match):
            call()
    x, u = torch.zeros(3, 50), torch.zeros(3)
    for kind, match, call in (
            (ValueError, "on a GPU", lambda: mnb.sample(x, u)),
            (ValueError, "on a GPU", lambda: mnb.sample(x, u, u, torch.ones(3, dtype=torch.int32), u, u)),
            (TypeError, "logits", lambda: mnb.sample(x.double(), u)),
            (TypeError, "u must", lambda: mnb.sample(x, u.double())),
            (ValueError, "u must", lambda: mnb.sample(x, u[:2])),
            (ValueError, "columns", lambda: mnb.sample(x[:, :0], u)),
            (TypeError, "temperature", lambda: mnb.sample(x, u, u.half())),
            (TypeError, "top_k", lambda: mnb.sample(x, u, 1.0, u)),
            (ValueError, "min_p", lambda: mnb.sample(x, u, min_p=u[:1])),
            (TypeError, "", lambda: mnb.sample(x, u, "hot")),
            (TypeError, "", lambda: mnb.sample(x, u, top_k=1.5)),
            (TypeError, "out", lambda: mnb.sample(x, u, out=u))):
        with pytest.raises(kind, match=match):
            call()


def test_rope_table():
    t = mnb.rope_table(100000, 64, base=1e6, device="cpu")
    assert np.abs(t.numpy() - dref.table(100000, 64, 1e6)).max() <= 2.0 ** -24
    f = torch.linspace(1, 0.01, 16)
    t = mnb.rope_table(10, 32, device="cpu", inv_freq=f)
    assert torch.equal(t[3, :16], torch.cos(3 * f.double()).float())
    with pytest.raises(ValueError):
        mnb.rope_table(10, 24)
    with pytest.raises(ValueError):
        mnb.rope_table(10, 32, inv_freq=f[:8])


# ------------------------------------------------------------------------------------------
# the references themselves
# ------------------------------------------------------------------------------------------


def test_reference_rotation_and_attention():
    r = np.random.default_rng(3)
    x = r.standard_normal((5, 2, 64))
    tab = dref.table(5, 64)
    for il in (False, True):
        y = dref.norm_rotate(x, None, 0, tab, il)
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-6) and np.array_equal(y[0], x[0])
        # scores depend on the distance of positions alone
        a = dref.norm_rotate(np.repeat(x[:1], 5, 0), None, 0, tab, il)
        b = dref.norm_rotate(np.repeat(x[1:2], 5, 0), None, 0, tab, il)
        assert np.allclose((a[1:] * b[:-1]).sum(-1), (a[1] * b[0]).sum(-1), atol=1e-5)
    q, k, v = r.standard_normal((3, 4, 64)), r.standard_normal((7, 2, 64)), r.standard_normal((7, 2, 64))
    t = [torch.from_numpy(z) for z in (q, k, v)]
    y, _ = dref.attention(q, k, v, 4, 0.2)
    s = torch.einsum("nhd,thd->hnt", t[0], t[1].repeat_interleave(2, 1)) * 0.2
    s = s.masked_fill(torch.arange(7)[None, None] > 4 + torch.arange(3)[None, :, None], -float("inf"))
    want = torch.einsum("hnt,thd->nhd", s.softmax(-1), t[2].repeat_interleave(2, 1))
    assert np.allclose(y, want.numpy())
    one, _ = dref.attention(q, k, v, 4, 0.2, window=1)
    assert np.allclose(one, v[4:7].repeat(2, 1))


def test_reference_sample():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    got = [dref.sample(x, u, 1.0, 0, 1.0, 0.0) for u in (0.0, 0.05, 0.11, 0.49, 0.51, 0.71, 0.95)]
    assert got == [0, 0, 1, 1, 2, 3, 4]
    assert [dref.sample(x, u, 1.0, 2, 1.0, 0.0) for u in (0.0, 0.6, 0.7)] == [1, 1, 2]     # the tie goes to the lower index
    assert [dref.sample(x, u, 1.0, 0, 0.55, 0.0) for u in (0.1, 0.9)] == [1, 2]
    assert {dref.sample(x, u, 1.0, 0, 1.0, 0.3) for u in np.linspace(0, 0.99, 50)} == {1, 2, 3}
    assert dref.sample(x, 0.99, 0.0, 0, 1.0, 0.0) == 1
