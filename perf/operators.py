"""The operators beside MatMulNBits, as calls to be timed: microscaled (MX) quantisation and product, the
root-mean-square norm with the residual's addition and MX output, and log probabilities over logits.

``listed()`` gives the cases, ``draw(rng)`` more of the same ranges, ``prepare(case, seed)`` what a program
has in hand before the call, ``run(state)`` one pass, ``work(case)`` the bytes and operations a pass cannot do
without, and ``exact(case, seed)`` the results from the definition in 64 bits.  With ``own`` false, ``run``
computes the operators from elementary torch operations in 32 bits; with ``own`` true it calls this
repository's kernels.

MX formats: blocks of 32 along the last axis share one power-of-two scale (E8M0, byte e stands for
2^(e - 127)); elements are FP4 (E2M1, two per byte, the even index in the low nibble) or FP8 (E4M3).  The
scale is 2^(floor(log2 max|x|) - emax), emax = 2 for FP4 and 8 for FP8; elements are rounded to nearest even
and clamped to the largest value (6 or 448).
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
EPS = 1e-6


def listed():
    return [
        # activations of a few decode rows on their way into an 8-bit product
        dict(name="quantise fp8 8x2048", op="quantise", m=8, k=2048, dtype="fp16", fmt="fp8"),
        # the tied lm_head's weight taken to 4 bits when a model is loaded, and read back
        dict(name="quantise fp4 49152x576", op="quantise", m=49152, k=576, dtype="bf16", fmt="fp4"),
        # one decode token through an MLP up-projection
        dict(name="product a8 1x8192x2048", op="product", m=1, n=8192, k=2048, act="fp8", dtype="fp16", bias=False),
        # eight sequences decoding together through the lm_head
        dict(name="product a8 8x49152x576", op="product", m=8, n=49152, k=576, act="fp8", dtype="fp16", bias=False),
        # a ragged batch: odd row and column counts, a last K block inside a tile, a bias
        dict(name="product a4 333x1000x1056", op="product", m=333, n=1000, k=1056, act="fp4", dtype="bf16", bias=True),
        # prefill of one prompt through an attention projection, 4 bits on both sides
        dict(name="product a4 1024x4096x4096", op="product", m=1024, n=4096, k=4096, act="fp4", dtype="fp16", bias=False),
        # the largest: batched prefill through an MLP projection, 8-bit activations
        dict(name="product a8 8192x9728x2560", op="product", m=8192, n=9728, k=2560, act="fp8", dtype="fp16", bias=False),
        # the norm in front of a decode projection
        dict(name="norm fp8 1x2048", op="norm", m=1, k=2048, dtype="fp16", out="fp8", residual=True),
        # a short prompt in a small model, 16 bits out
        dict(name="norm fp16 333x896", op="norm", m=333, k=896, dtype="fp16", out="same", residual=True),
        # batched prefill, quantised for the 8-bit product
        dict(name="norm fp8 8192x4096", op="norm", m=8192, k=4096, dtype="bf16", out="fp8", residual=True),
        # the token just sampled and its alternatives
        dict(name="logprobs 1x49152 top 5", op="logprobs", m=1, v=49152, dtype="fp16", top=5),
        # scoring every token of a prompt
        dict(name="logprobs 1024x49152 top 20", op="logprobs", m=1024, v=49152, dtype="fp16", top=20),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "norm", "logprobs"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "quantise":
        return dict(op=op, m=_spread(rng, 1, 8192), k=BLOCK * _spread(rng, 1, 128), dtype=rng.choice(["fp16", "bf16", "fp32"]),
                    fmt=rng.choice(["fp4", "fp8"]))
    if op == "product":
        # few rows (decode) as often as many (prefill)
        m = _spread(rng, 1, 32) if rng.random() < 0.5 else _spread(rng, 33, 4096)
        return dict(op=op, m=m, n=_spread(rng, 64, 16384), k=BLOCK * _spread(rng, 2, 160), act=rng.choice(["fp4", "fp8"]), dtype=dtype,
                    bias=rng.random() < 0.5)
    if op == "norm":
        out = rng.choice(["same", "fp4", "fp8"])
        k = _spread(rng, 64, 8192)
        return dict(op=op, m=_spread(rng, 1, 4096), k=k if out == "same" else BLOCK * max(1, k // BLOCK), dtype=dtype, out=out,
                    residual=rng.random() < 0.7)
    v = _spread(rng, 512, 262144)
    m = _spread(rng, 1, max(1, min(1024, (1 << 25) // v)))
    return dict(op=op, m=m, v=v, dtype=rng.choice(["fp16", "bf16", "fp32"]), top=rng.choice([0, 1, 5, 20]))


# ---- inputs ------------------------------------------------------------------------------------


def _randn(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _activations(gen, m, k, dtype):
    """Hidden states: normal values, a few channels many times larger, as trained models have them."""
    channel = torch.exp(0.5 * _randn(gen, (k,)))
    channel = torch.where(torch.rand((k,), generator=gen, device="cuda") < 0.01, 12.0 * channel, channel)
    return (_randn(gen, (m, k)) * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m = case["op"], case["m"]
    s = dict(case)
    if op == "quantise":
        s["x"] = _activations(gen, m, case["k"], DTYPES[case["dtype"]])
    elif op == "product":
        n, k = case["n"], case["k"]
        x = _quantise(_activations(gen, m, k, torch.float32), case["act"])
        w = _quantise(_randn(gen, (n, k), 0.02) * torch.exp(0.3 * _randn(gen, (n, 1))), "fp4")
        s["bias"] = _randn(gen, (n,), 0.5).to(DTYPES[case["dtype"]]) if case["bias"] else None
        if own:  # the weights in the kernels' layout, once, as a program that serves them keeps them
            import blockwise_bit_quantized_amd as mnb

            s["x"] = mnb.mx_tensor(x[0], x[1], _own_format(case["act"]))
            s["w"] = mnb.mx_pack(mnb.mx_tensor(w[0], w[1], mnb.MNB_MX_FP4))
        else:
            s["x"], s["w"] = x, w
    elif op == "norm":
        dtype = DTYPES[case["dtype"]]
        s["x"] = _activations(gen, m, case["k"], dtype)
        s["residual"] = _activations(gen, m, case["k"], dtype) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(gen, (case["k"],))).to(dtype)
    else:
        v = case["v"]
        # logits of a language model: a broad bulk, and a few tokens well above it in each row
        x = _randn(gen, (m, v), 2.0)
        at = torch.randint(0, v, (m, 8), generator=gen, device="cuda")
        x.scatter_add_(1, at, 4.0 + _randn(gen, (m, 8), 3.0))
        s["logits"] = x.to(DTYPES[case["dtype"]])
        tokens = torch.randint(0, v, (m,), generator=gen, device="cuda")
        likely = torch.rand((m,), generator=gen, device="cuda") < 0.7
        s["tokens"] = torch.where(likely, at[:, 0], tokens)
    return s


# ---- the plain form ----------------------------------------------------------------------------


def _power(e):
    """2^e in 32 bits for whole e in [-126, 127], from its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x, fmt):
    """(codes, scales) of x [m, k]: uint8 [m, k / 2] (FP4) or [m, k] (FP8), and uint8 [m, k / 32]."""
    m, k = x.shape
    v = x.float().view(m, k // BLOCK, BLOCK)
    amax = v.abs().amax(-1)
    e = torch.frexp(amax)[1].to(torch.int32) - 1 - (2 if fmt == "fp4" else 8)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    v = (v * _power((-e).clamp(-126, 127))[..., None]).view(m, k)
    scales = (e + 127).to(torch.uint8)
    if fmt == "fp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scales
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = torch.round(a / step) * step
    # the codes 0..7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6
    code = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, 2.0 + a, 4.0 + 0.5 * a)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def _dequantise(codes, scales, fmt):
    """The 32-bit values of (codes, scales)."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(FP4_VALUES, dtype=torch.float32, device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    m = scales.shape[0]
    v = v.reshape(m, -1, BLOCK)
    return (v * scales.view(torch.float8_e8m0fnu).float()[..., None]).view(m, -1)


def _mx_outputs(codes, scales, fmt, dtype):
    """A quantised tensor as the values it stands for: FP8 elements and their scales are number types of
    their own; FP4 elements have none, so they are read back."""
    if fmt == "fp8":
        return {"elements": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
    return {"values": _dequantise(codes, scales, fmt).to(dtype)}


def _run_plain(s):
    op = s["op"]
    if op == "quantise":
        return _mx_outputs(*_quantise(s["x"], s["fmt"]), s["fmt"], s["x"].dtype)
    if op == "product":
        y = _dequantise(*s["x"], s["act"]) @ _dequantise(*s["w"], "fp4").t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(DTYPES[s["dtype"]])}
    if op == "norm":
        dtype = s["x"].dtype
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        got = {"y": y.to(dtype)} if s["out"] == "same" else _mx_outputs(*_quantise(y, s["out"]), s["out"], dtype)
        if s["residual"] is not None:
            got["hidden"] = h.to(dtype)
        return got
    x = s["logits"].float()
    d = x - x.amax(-1, keepdim=True)
    p = torch.exp(d)
    total = p.sum(-1)
    lse = torch.log(total)
    got = {"logprob": d.gather(1, s["tokens"][:, None])[:, 0] - lse, "entropy": lse - (p * d).sum(-1) / total}
    if s["top"]:
        _, order = torch.sort(x, dim=-1, descending=True, stable=True)
        got["top_tokens"] = order[:, : s["top"]]
        got["top_logprobs"] = d.gather(1, got["top_tokens"]) - lse[:, None]
    return got


# ---- this repository's kernels -------------------------------------------------------------------


def _own_format(fmt):
    import blockwise_bit_quantized_amd as mnb

    return mnb.MNB_MX_FP4 if fmt == "fp4" else mnb.MNB_MX_FP8


def _own_outputs(mnb, q, dtype):
    if q.fmt == mnb.MNB_MX_FP8:
        return {"elements": q.codes.view(torch.float8_e4m3fn), "scales": q.scales.view(torch.float8_e8m0fnu)}
    return {"values": mnb.mx_dequantize(q, dtype)}


def _run_own(s):
    import blockwise_bit_quantized_amd as mnb

    op = s["op"]
    if op == "quantise":
        return _own_outputs(mnb, mnb.mx_quantize(s["x"], _own_format(s["fmt"])), s["x"].dtype)
    if op == "product":
        return {"y": mnb.mx_matmul(s["x"], s["w"], bias=s["bias"], dtype=DTYPES[s["dtype"]])}
    if op == "norm":
        fmt = None if s["out"] == "same" else _own_format(s["out"])
        r = mnb.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], fmt=fmt)
        got = {"y": r.y} if fmt is None else _own_outputs(mnb, r.q, s["x"].dtype)
        if s["residual"] is not None:
            got["hidden"] = r.hidden
        return got
    r = mnb.logprobs(s["logits"], s["tokens"], top=s["top"])
    got = {"logprob": r.logprob, "entropy": r.entropy}
    if s["top"]:
        got["top_tokens"], got["top_logprobs"] = r.top_tokens, r.top_logprobs
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------


def _mx_bytes(m, k, fmt):
    return m * k // (2 if fmt == "fp4" else 1) + m * (k // BLOCK)


def work(case):
    op, m = case["op"], case["m"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "quantise":
        k = case["k"]
        # the 4-bit cases read the values back too
        moved = m * k * size + _mx_bytes(m, k, case["fmt"])
        if case["fmt"] == "fp4":
            moved += m * k * size + _mx_bytes(m, k, case["fmt"])
        return {"bytes": moved, "flops": 3 * m * k}
    if op == "product":
        n, k = case["n"], case["k"]
        moved = _mx_bytes(m, k, case["act"]) + _mx_bytes(n, k, "fp4") + 2 * m * n + (2 * n if case["bias"] else 0)
        return {"bytes": moved, "flops": 2 * m * n * k}
    if op == "norm":
        k = case["k"]
        moved = 2 * m * k * (3 if case["residual"] else 1) + 2 * k
        if case["out"] == "same":
            moved += 2 * m * k
        else:
            moved += _mx_bytes(m, k, case["out"]) + (_mx_bytes(m, k, "fp4") + 2 * m * k if case["out"] == "fp4" else 0)
        return {"bytes": moved, "flops": 6 * m * k}
    v, top = case["v"], case["top"]
    return {"bytes": m * v * size + m * (8 + 8) + m * top * 12, "flops": 6 * m * v}


# ---- the definition in 64 bits -------------------------------------------------------------------


def _exact_power(e):
    """2^e in 64 bits for whole e in [-1022, 1023], from its bits (pow need not be exact, and ties are)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_elements(x, fmt):
    """(elements, scales) in 64 bits: every element the nearest value of its format (ties to the even one)."""
    m, k = x.shape
    b = x.double().reshape(m, k // BLOCK, BLOCK)
    top = b.abs().max(dim=2).values
    # the position of the highest bit, from the number's own exponent field; below every scale for zeros
    exponent = ((top.view(torch.int64) >> 52) - 1023).clamp(min=-200)
    scale = _exact_power((exponent - {"fp4": 2, "fp8": 8}[fmt]).clamp(-127, 127))
    q = b / scale[..., None]
    mantissa, lowest, largest = {"fp4": (1, 0, 6.0), "fp8": (3, -6, 448.0)}[fmt]
    size = q.abs().clamp(max=largest)
    octave = (size.view(torch.int64) >> 52) - 1023
    quantum = _exact_power(octave.clamp(min=lowest) - mantissa)
    q = torch.copysign(torch.round(size / quantum) * quantum, q)
    return q, scale


def _exact_mx(x, fmt):
    q, scale = _exact_elements(x, fmt)
    if fmt == "fp8":
        return {"elements": q.reshape(x.shape), "scales": scale}
    return {"values": (q * scale[..., None]).reshape(x.shape)}


def _exact_values(codes, scales, fmt):
    """64-bit values from the bits: sign, exponent and mantissa fields taken apart."""
    c = codes.long()
    if fmt == "fp4":
        c = torch.stack((c % 16, c // 16), -1).reshape(codes.shape[0], -1)
        sign, exp, man, bias, width = c // 8, (c // 2) % 4, c % 2, 1, 1
    else:
        sign, exp, man, bias, width = c // 128, (c // 8) % 16, c % 8, 7, 3
    fraction = man.double() / 2**width
    v = torch.where(exp > 0, (1 + fraction) * _exact_power(exp - bias), fraction * 2.0 ** (1 - bias))
    v = torch.where(sign > 0, -v, v)
    return v * _exact_power(scales.long() - 127).repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quantise":
        return _exact_mx(s["x"], case["fmt"])
    if op == "product":
        y = _exact_values(*s["x"], case["act"]) @ _exact_values(*s["w"], "fp4").transpose(0, 1).contiguous()
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if op == "norm":
        h = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
        y = s["weight"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["k"] + EPS)
        got = {"y": y} if case["out"] == "same" else _exact_mx(y, case["out"])
        if s["residual"] is not None:
            got["hidden"] = h
        return got
    x = s["logits"].double()
    logp = x - torch.logsumexp(x, dim=1, keepdim=True)
    got = {"logprob": logp[torch.arange(case["m"], device=x.device), s["tokens"]], "entropy": -(logp.exp() * logp).sum(1)}
    if case["top"]:
        # one whole number a token orders by value, then by the lower index
        bits = s["logits"].float().view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 20) - torch.arange(case["v"], device=x.device)
        got["top_tokens"] = torch.topk(key, case["top"], dim=1, sorted=True).indices
        got["top_logprobs"] = logp.gather(1, got["top_tokens"])
    return got
