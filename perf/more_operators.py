"""The operators of a decoding step around the attention and behind the logits, as calls to be timed: queries, keys
and values on their way into a paged cache held in 4 bits (norms for each head, rotation, quantisation), attention over
that cache, and the choice of the next token.

``listed()`` gives the cases, ``draw(rng)`` more of the same ranges, ``prepare(case, seed)`` what a program
has in hand before the call, ``run(state)`` one pass, ``work(case)`` the bytes and operations a pass cannot do
without, and ``exact(case, seed)`` the results from the definition in 64 bits.  With ``own`` false, ``run``
computes the operators from elementary torch operations; with ``own`` true it calls this repository's kernels.

A sequence b has ``lengths[b]`` tokens in the cache after the call, its new ones last.  Page ``pages[b, p // page]``
holds position p.  A row of an idle sequence (of length 0) has no position; its results are zeros.  Keys and values are MX FP4 along the head: 32 elements share one power of two, 2^(floor(log2
max|x|) - 2); elements are E2M1, rounded to nearest even and clamped to 6.
"""
import math
import random

import torch

own = False

BLOCK = 32
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
EPS = 1e-6
ROPE_BASE = 10000.0

# query heads, key/value heads, elements of a head
SMALL, MIDDLE, LARGE, WIDE, ODD, EQUAL = (9, 3, 64), (14, 2, 64), (32, 8, 128), (8, 1, 256), (20, 4, 96), (16, 16, 128)


def _cache_case(op, name, heads, batch, new, length, page, dtype, ragged=False, window=0, norm=True, rope="half", **more):
    case = dict(op=op, hq=heads[0], hkv=heads[1], d=heads[2], batch=batch, new=new, length=length, page=page, dtype=dtype,
                ragged=ragged, **more)
    case.update(dict(window=window) if op == "attention" else dict(norm=norm, rope=rope))
    return dict(name=name, **case) if name else case


def listed():
    c = _cache_case
    return [
        # one token of one sequence in a small model: latency alone
        c("append", "append 1 token 9/3x64", SMALL, 1, 1, 700, 32, "fp16", norm=False),
        # a batch of decoding sequences of different lengths, with norms of queries and keys
        c("append", "append 64 tokens 32/8x128", LARGE, 64, 1, 4096, 64, "bf16", ragged=True),
        # a long prompt, or many short ones, being taken in
        c("append", "append 8192 tokens 32/8x128", LARGE, 2, 4096, 4096, 64, "bf16"),
        # one sequence decoding in a small model
        c("attention", "attention 1x1 over 700 14/2x64", MIDDLE, 1, 1, 700, 32, "fp16"),
        # a served batch: every sequence of its own length, one place of the batch idle
        c("attention", "attention 32x1 over 4096 32/8x128", LARGE, 32, 1, 4096, 64, "bf16", ragged=True),
        # one sequence decoding behind a very long document
        c("attention", "attention 1x1 over 131072 32/8x128", LARGE, 1, 1, 131072, 256, "bf16"),
        # a few drafted tokens of each sequence verified at once, a sliding window
        c("attention", "attention 8x5 over 2001 20/4x96", ODD, 8, 5, 2001, 16, "fp16", ragged=True, window=1024),
        # the next part of prompts that are taken in by parts, odd sizes
        c("attention", "attention 4x333 over 3001 14/2x64", MIDDLE, 4, 333, 3001, 64, "fp16", ragged=True),
        # the largest: a whole prompt at once
        c("attention", "attention 1x8192 over 8192 32/8x128", LARGE, 1, 8192, 8192, 64, "bf16"),
        # the next token of one sequence, the usual filters
        dict(name="sample 1x49152 all filters", op="sample", m=1, v=49152, dtype="fp16", filters="all"),
        # a served batch, each row with filters of its own
        dict(name="sample 64x131072 own filters", op="sample", m=64, v=131072, dtype="bf16", filters="rows"),
        # many samples of a prompt: the whole distribution
        dict(name="sample 1024x49152 temperature", op="sample", m=1024, v=49152, dtype="fp16", filters="none"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "sample"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "sample":
        v = _spread(rng, 512, 262144)
        return dict(op=op, m=_spread(rng, 1, max(1, min(1024, (1 << 24) // v))), v=v, dtype=rng.choice(["fp16", "bf16", "fp32"]),
                    filters=rng.choice(["none", "all", "rows"]))
    heads = rng.choice([SMALL, MIDDLE, LARGE, WIDE, ODD, EQUAL])
    page = rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["one", "few", "many"])
    if op == "append":
        new = {"one": 1, "few": rng.randint(2, 8), "many": _spread(rng, 16, 2048)}[kind]
        batch = _spread(rng, 1, max(1, min(128, 8192 // new)))
        return _cache_case(op, None, heads, batch, new, new + _spread(rng, 1, 8192), page, dtype, ragged=rng.random() < 0.6,
                           norm=rng.random() < 0.6, rope=rng.choice(["half", "pairs", "part"]))
    new = {"one": 1, "few": rng.randint(2, 8), "many": _spread(rng, 16, 2048)}[kind]
    length = new + _spread(rng, 1, 32768 if kind == "one" else 8192 if kind == "few" else 2048)
    budget = (1 << 17) if kind != "many" else 8192          # tokens of all caches together
    batch = _spread(rng, 1, max(1, min(64, budget // length)))
    return _cache_case(op, None, heads, batch, new, length, page, dtype, ragged=rng.random() < 0.6,
                       window=rng.choice([0, 0, _spread(rng, 16, 4096)]))


# ---- inputs ------------------------------------------------------------------------------------


def _sizes(case):
    """(lengths, new tokens) of the sequences, from the case alone."""
    batch, new, length = case["batch"], case["new"], case["length"]
    if not case["ragged"]:
        return [length] * batch, [new] * batch
    rng = random.Random(length * 1009 + batch * 31 + new)
    count = [rng.randint((new + 1) // 2, new) for _ in range(batch)]
    total = [max(n, rng.randint(length // 4, length)) for n in count]
    total[0], count[0] = length, new
    if batch >= 4:                     # an idle place of the batch
        total[-1] = 0
        count[-1] = 1 if new == 1 else 0
    return total, count


def _randn(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _table(n, rot):
    """cos | sin of the angles of n positions, fp32 [n, rot]; the angles in 64 bits."""
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _heads(gen, n, heads, d, dtype):
    """Rows of heads as projections give them: normal values, a few channels several times larger."""
    channel = torch.exp(0.3 * _randn(gen, (heads, d)))
    channel = torch.where(torch.rand((heads, d), generator=gen, device="cuda") < 0.02, 4.0 * channel, channel)
    return (_randn(gen, (n, heads, d)) * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "sample":
        return _prepare_sample(s, gen)
    dtype, hq, hkv, d, page = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"], case["page"]
    lengths, count = _sizes(case)
    batch, width = len(lengths), -(-case["length"] // page)
    used = batch * width
    order = torch.randperm(used + 3, generator=gen, device="cuda")[:used].view(batch, width).to(torch.int32)
    rows = sum(count)
    starts = [0]
    for n in count:
        starts.append(starts[-1] + n)
    s.update(lengths_host=lengths, count_host=count, starts_host=starts, rows=rows, pages=order, lengths=_ints(lengths),
             starts=None if case["new"] == 1 else _ints(starts))
    if case["op"] == "append":
        # the slices of one projection's output
        wide = _heads(gen, rows, hq + 2 * hkv, d, dtype)
        s["q"], s["k"], s["v"] = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:]
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1.0 + 0.2 * _randn(gen, (d,))).to(dtype) for _ in range(2))
        s["table"] = _table(width * page, d // 2 if case["rope"] == "part" else d)
        s["cache"] = _empty_cache(used + 3, hkv, page, d)
        return s
    s["q"] = _heads(gen, rows, hq, d, dtype)
    total = sum(lengths)
    k, v = _heads(gen, total, hkv, d, dtype), _heads(gen, total, hkv, d, dtype)
    s["cache"] = _empty_cache(used + 3, hkv, page, d)
    whole = [0]
    for n in lengths:
        whole.append(whole[-1] + n)
    if own:
        import blockwise_bit_quantized_amd as mnb

        mnb.kv_append(None, k, v, s["cache"], s["pages"], s["lengths"], starts=_ints(whole))
    else:
        _store(s["cache"], k, v, *_places(s, lengths, lengths))
    return s


def _prepare_sample(s, gen):
    m, v = s["m"], s["v"]
    # logits of a language model: a broad bulk, and a few tokens well above it in each row
    x = _randn(gen, (m, v), 2.0)
    at = torch.randint(0, v, (m, 8), generator=gen, device="cuda")
    x.scatter_add_(1, at, 4.0 + _randn(gen, (m, 8), 3.0))
    s["logits"] = x.to(DTYPES[s["dtype"]])
    s["u"] = torch.rand((m,), generator=gen, device="cuda", dtype=torch.float32)
    if s["filters"] == "rows":
        def pick(values, dtype):
            at = torch.randint(0, len(values), (m,), generator=gen, device="cuda")
            return torch.tensor(values, device="cuda", dtype=dtype)[at]
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.3], torch.float32)
        s["top_k"] = pick([0, 1, 20, 50, 1000], torch.int32)
        s["top_p"] = pick([1.0, 0.9, 0.95, 0.5], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.05, 0.1], torch.float32)
    elif s["filters"] == "all":
        s.update(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    else:
        s.update(temperature=0.9, top_k=0, top_p=1.0, min_p=0.0)
    return s


def _empty_cache(pages, hkv, page, d):
    if own:
        import blockwise_bit_quantized_amd as mnb

        return mnb.kv_cache(pages, hkv, d, page_size=page, device="cuda")
    return {w + part: torch.zeros((pages, hkv, page, d // per), dtype=torch.uint8, device="cuda")
            for w in "kv" for part, per in (("_codes", 2), ("_scales", BLOCK))}


def _places(s, lengths, count):
    """(page, place in it) of the last count[b] tokens of every sequence, in order."""
    b = torch.cat([torch.full((n,), i, dtype=torch.long) for i, n in enumerate(count)]).cuda()
    p = torch.cat([torch.arange(t - n, t) for t, n in zip(lengths, count)]).cuda()
    there = p >= 0
    return s["pages"][b, (p.clamp(min=0) // s["page"])].long(), p.clamp(min=0) % s["page"], p, there


# ---- the plain form ----------------------------------------------------------------------------


def _power(e):
    """2^e in 32 bits for whole e in [-126, 127], from its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x):
    """(codes, scales) of x [..., d]: uint8 [..., d / 2] and [..., d / 32]."""
    d = x.shape[-1]
    v = x.float().reshape(*x.shape[:-1], d // BLOCK, BLOCK)
    amax = v.abs().amax(-1)
    e = torch.frexp(amax)[1].to(torch.int32) - 3
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    v = (v * _power((-e).clamp(-126, 127))[..., None]).reshape(x.shape)
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = torch.round(a / step) * step
    # the codes 0..7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6
    code = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, 2.0 + a, 4.0 + 0.5 * a)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _dequantise(codes, scales):
    """The 32-bit values of (codes, scales)."""
    table = torch.tensor(FP4_VALUES, dtype=torch.float32, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(*scales.shape, BLOCK) * scales.view(torch.float8_e8m0fnu).float()[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _store(cache, k, v, page, place, p, there):
    for name, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x)
        cache[name + "_codes"][page[there], :, place[there]] = codes[there]
        cache[name + "_scales"][page[there], :, place[there]] = scales[there]


def _rotate(x, cos, sin, rope):
    """The first 2 * cos.shape[-1] elements of every head rotated, in pairs (i, i + half) or (2i, 2i + 1)."""
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if rope == "pairs":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rot:]), -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)


def _run_plain_append(s):
    page, place, p, there = _places(s, s["lengths_host"], s["count_host"])
    at = s["table"][p.clamp(min=0)]
    cos, sin = at.chunk(2, -1)
    out = {}
    for name, wide in (("q", torch.float32), ("k", torch.float64)):
        # keys in 64 bits: 32 would put values next to a border of the 4-bit grid on either side
        x = s[name].to(wide)
        if s[name + "_weight"] is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[name + "_weight"].to(wide)
        out[name] = torch.where(there[:, None, None], _rotate(x, cos.to(wide), sin.to(wide), s["rope"]), 0.0)
    dtype = s["q"].dtype
    _store(s["cache"], _toward_odd(out["k"]), s["v"], page, place, p, there)
    got, c = {"q": out["q"].to(dtype)}, s["cache"]
    for name in "kv":
        x = _dequantise(c[name + "_codes"][page, :, place], c[name + "_scales"][page, :, place])
        got[name] = torch.where(there[:, None, None], x, 0.0).to(dtype)
    return got


def _toward_odd(x):
    """64 bits to 32, inexact values to the neighbour whose last bit is odd: a later rounding to fewer bits is then that of x."""
    f = x.float()
    bits = f.view(torch.int32)
    bits = torch.where(f.double().abs() > x.abs(), bits - 1, bits)
    return torch.where(f.double() == x, bits, bits | 1).view(torch.float32)


def _visible(n, total, window):
    """bool [n, total]: what the last n of total tokens see."""
    p = torch.arange(total - n, total, device="cuda")[:, None]
    t = torch.arange(total, device="cuda")[None]
    return (t <= p) & (t > p - window) if window else t <= p


def _run_plain_attention(s):
    hq, hkv, d, c = s["hq"], s["hkv"], s["d"], s["cache"]
    y = torch.zeros_like(s["q"])
    for b, (total, n) in enumerate(zip(s["lengths_host"], s["count_host"])):
        if total == 0 or n == 0:
            continue
        p = torch.arange(total, device="cuda")
        page, place = s["pages"][b, p // s["page"]].long(), p % s["page"]
        k = _dequantise(c["k_codes"][page, :, place], c["k_scales"][page, :, place]).permute(1, 2, 0).contiguous()
        v = _dequantise(c["v_codes"][page, :, place], c["v_scales"][page, :, place]).permute(1, 0, 2).contiguous()
        at = slice(s["starts_host"][b], s["starts_host"][b] + n)
        q = s["q"][at].float().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
        x = torch.matmul(q, k).view(hkv, hq // hkv, n, total) * (d ** -0.5)
        x = torch.where(_visible(n, total, s["window"]), x, -math.inf)
        x = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.matmul(x.view(hkv, -1, total), v).view(hkv, hq // hkv, n, d) / x.sum(-1, keepdim=True)
        y[at] = o.permute(2, 0, 1, 3).reshape(n, hq, d).to(y.dtype)
    return {"y": y}


def _run_plain_sample(s):
    x = s["logits"].double()
    m, v = x.shape

    def column(name, dtype):
        return torch.as_tensor(s[name], device="cuda", dtype=torch.float32 if dtype is torch.float64 else dtype).to(dtype).expand(m)[:, None]
    t, k, top_p, min_p = (column(n, d) for n, d in (("temperature", torch.float64), ("top_k", torch.int64), ("top_p", torch.float64),
                                                    ("min_p", torch.float64)))
    greedy = t == 0
    values, order = torch.sort(x, dim=-1, descending=True, stable=True)
    p = torch.exp((values - values[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(v, device="cuda")
    keep = (k <= 0) | (rank < k)
    p = torch.where(keep, p, 0.0)
    before = torch.cumsum(p, -1) - p
    keep = keep & ((top_p >= 1.0) | (before < top_p * p.sum(-1, keepdim=True))) & (p >= min_p)
    keep[:, 0] = True
    weight = torch.zeros_like(x).scatter_(1, order, torch.where(keep, p, 0.0))
    total = torch.cumsum(weight, -1)
    token = torch.searchsorted(total, s["u"].double()[:, None] * total[:, -1:], right=True)
    return {"tokens": torch.where(greedy, order[:, :1], token.clamp(max=v - 1))[:, 0]}


def _run_plain(s):
    return {"append": _run_plain_append, "attention": _run_plain_attention, "sample": _run_plain_sample}[s["op"]](s)


# ---- this repository's kernels -------------------------------------------------------------------


def _run_own(s):
    import blockwise_bit_quantized_amd as mnb

    if s["op"] == "sample":
        return {"tokens": mnb.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                     min_p=s["min_p"])}
    if s["op"] == "attention":
        return {"y": mnb.kv_attention(s["q"], s["cache"], s["pages"], s["lengths"], starts=s["starts"], window=s["window"])}
    q = mnb.kv_append(s["q"], s["k"], s["v"], s["cache"], s["pages"], s["lengths"], starts=s["starts"], rope=s["table"],
                      q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["rope"] == "pairs")
    k, v = mnb.kv_read(s["cache"], s["pages"], s["lengths"], s["rows"], starts=s["starts"], dtype=s["q"].dtype)
    return {"q": q, "k": k, "v": v}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    if case["op"] == "sample":
        m, v = case["m"], case["v"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": m * v * size + m * (4 + 8) + (m * 16 if case["filters"] == "rows" else 0), "flops": 6 * m * v}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lengths, count = _sizes(case)
    rows, token = sum(count), 2 * hkv * (d // 2 + d // BLOCK)      # bytes of a token in the cache
    if case["op"] == "append":
        rot = d // 2 if case["rope"] == "part" else d
        # the new rows are read back from the cache too
        return {"bytes": rows * (4 * hq * d + 4 * hkv * d + 4 * rot + 2 * token + 4 * hkv * d) + 4 * d * bool(case["norm"]),
                "flops": 10 * rows * (hq + hkv) * d}
    window, read, pairs = case["window"], 0, 0
    for total, n in zip(lengths, count):
        n = min(n, total)
        if n == 0:
            continue
        first = max(0, total - n - window + 1) if window else 0
        read += total - first
        seen = [min(p + 1, window) if window else p + 1 for p in (total - n, total - 1)]
        pairs += sum(min(p + 1, window) for p in range(total - n, total)) if window else n * (seen[0] + seen[1]) // 2
    return {"bytes": read * token + 4 * rows * hq * d, "flops": 4 * hq * d * pairs}


# ---- the definition in 64 bits -------------------------------------------------------------------


def _exact_power(e):
    """2^e in 64 bits for whole e in [-1022, 1023], from its bits (pow need not be exact, and ties are)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx(x):
    """x [..., d] as the values its FP4 form stands for: every element the nearest of its grid, ties to the even one."""
    b = x.double().reshape(-1, BLOCK)
    top = b.abs().max(dim=1).values
    # the position of the highest bit, from the number's own exponent field; below every scale for zeros
    exponent = ((top.view(torch.int64) >> 52) - 1023).clamp(min=-200)
    scale = _exact_power((exponent - 2).clamp(-127, 127))[:, None]
    size = (b / scale).abs().clamp(max=6.0)
    octave = (size.view(torch.int64) >> 52) - 1023
    quantum = _exact_power(octave.clamp(min=0) - 1)
    return (torch.copysign(torch.round(size / quantum) * quantum, b) * scale).reshape(x.shape)


def _exact_sample(s):
    # one whole number a token orders by value, then by the lower index
    bits = s["logits"].float().view(torch.int32).long()
    v = bits.shape[1]
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 20) - torch.arange(v, device="cuda")
    got = []
    for r in range(bits.shape[0]):
        t, k, top_p, min_p = (float(torch.as_tensor(s[n], dtype=torch.float32).reshape(-1).expand(bits.shape[0])[r].item())
                              for n in ("temperature", "top_k", "top_p", "min_p"))
        order = torch.argsort(key[r], descending=True)
        if t == 0.0:
            got.append(order[0])
            continue
        if k > 0:
            order = order[:int(k)]
        z = s["logits"][r].double()[order] / t
        p = torch.softmax(z, 0)
        if top_p < 1.0:
            # the smallest prefix that reaches top_p
            n = int((torch.cumsum(p, 0) < top_p).sum().item()) + 1
            order, p = order[:n], p[:n]
        p = p / p[0]
        stay = p >= min_p
        stay[0] = True
        kept, place = torch.sort(order[stay])
        c = torch.cumsum(p[stay][place], 0)
        at = int((c <= s["u"][r].double() * c[-1]).sum().item())
        got.append(kept[min(at, len(kept) - 1)])
    return {"tokens": torch.stack(got)}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "sample":
        return _exact_sample(s)
    hq, hkv, d, count, lengths = case["hq"], case["hkv"], case["d"], s["count_host"], s["lengths_host"]
    if case["op"] == "append":
        at = torch.cat([torch.arange(t - n, t) for t, n in zip(lengths, count)]).cuda()
        there = (at >= 0)[:, None, None]
        angle = s["table"].double()[at.clamp(min=0)]
        half = angle.shape[1] // 2
        turn = torch.complex(angle[:, None, :half], angle[:, None, half:])
        done = {}
        for name in "qk":
            x, w = s[name].double(), s[name + "_weight"]
            if w is not None:
                x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
            if case["rope"] == "pairs":
                z = turn * torch.complex(x[..., 0:2 * half:2].contiguous(), x[..., 1:2 * half:2].contiguous())
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = turn * torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous())
                head = torch.cat((z.real, z.imag), -1)
            done[name] = torch.cat((head, x[..., 2 * half:]), -1)
        return {"q": torch.where(there, done["q"], 0.0), "k": torch.where(there, _exact_mx(done["k"]), 0.0), "v": torch.where(there, _exact_mx(s["v"]), 0.0)}
    # keys and values anew from the generator, as prepare drew them, rounded by the format's definition
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, width = DTYPES[case["dtype"]], -(-case["length"] // case["page"])
    torch.randperm(len(lengths) * width + 3, generator=gen, device="cuda")
    q = _heads(gen, s["rows"], hq, d, dtype).double()
    k, v = _heads(gen, sum(lengths), hkv, d, dtype), _heads(gen, sum(lengths), hkv, d, dtype)
    y = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device="cuda")
    first = 0
    for b, (total, n) in enumerate(zip(lengths, count)):
        if total and n:
            kb, vb = _exact_mx(k[first:first + total]), _exact_mx(v[first:first + total])
            r0, p = s["starts_host"][b], torch.arange(total - n, total, device="cuda")[:, None]
            behind = p - torch.arange(total, device="cuda")[None]
            hidden = (behind < 0) | ((behind >= case["window"]) if case["window"] else (behind < 0))
            for h in range(hq):
                kh, vh = kb[:, h // (hq // hkv)], vb[:, h // (hq // hkv)]
                logit = (q[r0:r0 + n, h] @ kh.t().contiguous()) / math.sqrt(d)
                logit.masked_fill_(hidden, -math.inf)
                y[r0:r0 + n, h] = torch.softmax(logit, -1) @ vh.contiguous()
        first += total
    return {"y": y}
