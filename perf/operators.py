"""Workloads of the MXFP4 operators: what is measured, in plain torch and through the library.

``run(state)`` is one pass. With ``own`` false it is the plain form: elementary torch
operations in fp32 (fp64 next to a rounding border), rounded once at the end. With
``own`` true it is the calls a user of the library makes.

Kinds of case:

* ``quantize``  bf16 [m, k] -> MXFP4 -> read back as bf16
* ``swiglu``    gate, up [m, k] -> SwiGLU -> MXFP4 -> read back as bf16
* ``gemm``      the product of an MXFP4 activation [m, k] and weight [n, k] in hand
* ``linear``    bf16 [m, k] quantized, then multiplied by an MXFP4 weight [n, k]
* ``cache``     new keys and values appended to a paged MXFP4 cache and read back
* ``attend``    attention of new queries over a paged MXFP4 cache
"""
import torch

own = False

BLOCK = 32
PAGE_SPARE = 3  # pages of a cache that belong to no sequence


def _lib():
    import nvfp4_block_scaled_swiglu_amd as nv
    return nv


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one token's QKV activation: launch latency
        {"name": "quantize_token", "kind": "quantize", "m": 1, "k": 5376},
        # the FC2 producer on a ragged row count of the video sweep
        {"name": "swiglu_fc2", "kind": "swiglu", "m": 37711, "k": 14336},
        # one token through FC2: the weight is read once, nothing else counts
        {"name": "gemm_token", "kind": "gemm", "m": 1, "n": 5376, "k": 14336},
        # a decoding batch through QKV
        {"name": "gemm_batch", "kind": "gemm", "m": 48, "n": 16128, "k": 5376},
        # the canonical FC2 product
        {"name": "gemm_fc2", "kind": "gemm", "m": 37810, "n": 5376, "k": 14336},
        # a short prompt through the attention-output projection, quantized on the way
        {"name": "linear_out", "kind": "linear", "m": 1021, "n": 5376, "k": 7168},
        # a decoding batch writes one token a sequence
        {"name": "cache_token", "kind": "cache", "batch": 48, "q": 1, "kv": 1500, "kv_heads": 8, "dim": 128, "page": 16},
        # ragged prompts written whole
        {"name": "cache_prompt", "kind": "cache", "batch": 5, "q": 8191, "kv": 8191, "kv_heads": 8, "dim": 128,
         "page": 64},
        # single tokens of a ragged decoding batch, 7 query heads on each kv head
        {"name": "attend_decode", "kind": "attend", "batch": 48, "q": 1, "kv": 8200, "heads": 56, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0, "sinks": 0},
        # one sequence, one token, a long cache: few rows, the work is split over the cache
        {"name": "attend_long", "kind": "attend", "batch": 1, "q": 1, "kv": 131071, "heads": 32, "kv_heads": 4,
         "dim": 128, "page": 16, "window": 0, "sinks": 0},
        # a prompt with a sliding window and first tokens that stay visible, small heads
        {"name": "attend_window", "kind": "attend", "batch": 2, "q": 3001, "kv": 6000, "heads": 32, "kv_heads": 8,
         "dim": 64, "page": 32, "window": 1024, "sinks": 5},
        # a prompt chunk after a cached prefix
        {"name": "attend_prompt", "kind": "attend", "batch": 2, "q": 4096, "kv": 6200, "heads": 56, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0, "sinks": 0},
    ]


def _log(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["quantize", "swiglu", "gemm", "gemm", "linear", "cache", "attend", "attend", "attend"])
    if kind in ("quantize", "swiglu"):
        return {"kind": kind, "m": _log(rng, 1, 37810), "k": BLOCK * _log(rng, 2, 448)}
    if kind in ("gemm", "linear"):
        return {"kind": kind, "m": _log(rng, 1, 37810), "n": _log(rng, 64, 5376), "k": BLOCK * _log(rng, 8, 448)}
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if kind == "cache":
        q = rng.choice([1, _log(rng, 1, 8191)])
        return {"kind": kind, "batch": _log(rng, 1, 48) if q < 512 else rng.randint(1, 5), "q": q,
                "kv": _log(rng, q, max(q, 8191)), "kv_heads": kv_heads, "dim": dim, "page": page}
    form = rng.choice(["decode", "long", "prompt"])
    heads = kv_heads * rng.choice([1, 3, 4, 7])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, 2048), rng.choice([0, 1, 4, 63]))])
    if form == "decode":
        batch, q, kv = _log(rng, 2, 48), rng.choice([1, 1, 2, 5]), _log(rng, 16, 8200)
    elif form == "long":
        batch, q, kv = 1, 1, _log(rng, 8192, 131071)
    else:
        batch, q = rng.choice([1, 2]), _log(rng, 64, 4096)
        kv = _log(rng, q, 6200)
    return {"kind": "attend", "batch": batch, "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "window": window, "sinks": sinks}


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: ragged, the first the longest."""
    b = case["batch"]
    kv = [max(1, case["kv"] - i * (case["kv"] // (2 * b))) for i in range(b)]
    q = [min(kv[i], max(1, case["q"] - i * (case["q"] // (3 * b)))) for i in range(b)]
    return q, kv


def _pairs(case):
    """(query, visible token) pairs of one head, and the tokens that some query of their sequence sees."""
    pairs = tokens = 0
    w, s = case["window"], case["sinks"]
    for q, kv in zip(*_lengths(case)):
        low = max(0, kv - q - w + 1) if w else 0
        tokens += kv - low + min(s, low)
        p = torch.arange(kv - q, kv, dtype=torch.int64)
        n = p + 1
        if w:
            n = torch.minimum(n, torch.full_like(n, w)) + torch.minimum((p - w + 1).clamp(min=0),
                                                                       torch.full_like(n, s))
        pairs += int(n.sum())
    return pairs, tokens


def work(case):
    kind = case["kind"]
    packed = 0.5 + 1 / BLOCK  # bytes of an MXFP4 element with its share of a scale
    if kind in ("quantize", "swiglu"):
        e = case["m"] * case["k"]
        return {"bytes": e * ((4 if kind == "swiglu" else 2) + packed + packed + 2),
                "flops": e * (8 if kind == "swiglu" else 3)}
    if kind in ("gemm", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        a = m * k * (packed if kind == "gemm" else 2 + 2 * packed)
        return {"bytes": a + n * k * packed + 2 * m * n, "flops": 2 * m * n * k}
    q, kv = _lengths(case)
    if kind == "cache":
        e = 2 * sum(q) * case["kv_heads"] * case["dim"]
        return {"bytes": e * (2 + packed + packed + 2), "flops": 3 * e}
    pairs, tokens = _pairs(case)
    return {"bytes": 2 * tokens * case["kv_heads"] * case["dim"] * packed + 4 * sum(q) * case["heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---- inputs --------------------------------------------------------------------------------

def _normal(shape, seed, sigma=1.0, outliers=False):
    """bf16 N(0, sigma); with outliers every 100th channel is 20 times as large, as in the block's activations."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, sigma, generator=g)
    if outliers:
        x[..., 7::100] *= 20
    return x


def _paged(case, seed):
    """New tokens' k and v, the cached tokens before them, and where each sequence's pages are."""
    q, kv = _lengths(case)
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    most = -(-max(kv) // page)
    count = sum(-(-n // page) for n in kv)
    g = torch.Generator(device="cuda").manual_seed(seed + 11)
    order = torch.randperm(count + PAGE_SPARE, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(kv):
        pages = -(-n // page)
        table[i, :pages] = order[at:at + pages]
        at += pages
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    starts = lambda n: torch.tensor([0] + n, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
    return {"table": table, "lens": lens, "starts": starts(q), "all_starts": starts(kv), "pages": count + PAGE_SPARE,
            "tokens": sum(q), "longest": max(kv), "most": max(q)}, (h, d, page, sum(q), sum(kv))


def _inputs(case, seed):
    """The bf16 tensors of a case, from its seed alone."""
    kind = case["kind"]
    if kind == "quantize":
        return {"x": _normal((case["m"], case["k"]), seed, outliers=True)}
    if kind == "swiglu":
        return {"gate": _normal((case["m"], case["k"]), seed, outliers=True),
                "up": _normal((case["m"], case["k"]), seed + 1)}
    if kind in ("gemm", "linear"):
        return {"x": _normal((case["m"], case["k"]), seed, outliers=True),
                "w": _normal((case["n"], case["k"]), seed + 1, 0.02)}
    plan, (h, d, page, new, cached) = _paged(case, seed)
    plan["page"] = page
    if kind == "cache":
        return dict(plan, k=_normal((new, h, d), seed, outliers=True), v=_normal((new, h, d), seed + 1))
    return dict(plan, q=_normal((new, case["heads"], d), seed + 2),
                k=_normal((cached, h, d), seed, outliers=True), v=_normal((cached, h, d), seed + 1))


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    kind = case["kind"]
    if kind in ("gemm", "linear"):
        w, x = s.pop("w"), s["x"]
        if own:
            s["w"] = _lib().mxfp4_quantize(w)
            if kind == "gemm":
                s["x"] = _lib().mxfp4_quantize(x)
        else:
            s["w"] = _rounded(w)
            if kind == "gemm":
                s["x"] = _rounded(x)
    elif kind in ("cache", "attend"):
        shape = (s["pages"], case["kv_heads"], case["page"], case["dim"])
        if own:
            s["cache"] = _lib().empty_mxfp4_cache(s["pages"], case["page"], case["kv_heads"], case["dim"], "cuda")
            if kind == "attend":
                _lib().mxfp4_cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["all_starts"])
        else:
            s["cache"] = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            if kind == "attend":
                _append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["all_starts"])
        if kind == "attend":
            s["scale"] = case["dim"] ** -0.5
            del s["k"], s["v"]
    return s


# ---- the plain form ------------------------------------------------------------------------

def _two(e):
    """2^e in fp32 for whole -127 <= e <= 127, by its bits (a power function may be an ulp off)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _rounded(x):
    """x rounded to MXFP4, as the bf16 values that the codes and scales stand for."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(min=-127)
    a = b.abs() * _two(-e)
    m = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5)
    return (torch.copysign(m, b) * _two(e)).flatten(-2).to(torch.bfloat16)


def _swiglu(gate, up):
    """RN_bf16(silu_bf16(gate) * up). silu in 64 bits, and its rounding to fp32 on the way to bf16 kept off the ties."""
    g = gate.double()
    s = g / (1 + torch.exp(-g))
    f = s.float()
    bits = f.view(torch.int32)
    tie = (bits & 0xFFFF) == 0x8000
    off = (s.abs() > f.double().abs()).int() - (s.abs() < f.double().abs()).int()
    silu = (bits + tie * off).view(torch.float32).to(torch.bfloat16)
    return (silu.float() * up.float()).to(torch.bfloat16)


def _places(table, lens, starts, page, count):
    """(page, slot in it) of each new token: the last starts[b + 1] - starts[b] positions of sequence b."""
    row = torch.arange(count, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    at = lens[seq].long() - starts[seq + 1] + row
    return table[seq, at // page].long(), at % page


def _append(cache, k, v, table, lens, starts):
    page, slot = _places(table, lens, starts, cache[0].shape[2], k.shape[0])
    cache[0][page, :, slot] = _rounded(k)
    cache[1][page, :, slot] = _rounded(v)


def _read(cache, table, lens, starts, count):
    page, slot = _places(table, lens, starts, cache[0].shape[2], count)
    return cache[0][page, :, slot], cache[1][page, :, slot]


def _attend(s):
    case = s["case"]
    h, d = case["kv_heads"], case["dim"]
    g, b = case["heads"] // h, case["batch"]
    table = s["table"].long().clamp(min=0)
    k, v = (c[table].transpose(1, 2).flatten(2, 3).float() for c in s["cache"])  # [b, h, tokens, d]
    t = torch.arange(k.shape[2], device="cuda")
    v = torch.where((t < s["lens"][:, None])[:, None, :, None], v, 0.0)
    count = s["starts"][1:] - s["starts"][:-1]
    row = torch.arange(s["most"], device="cuda")
    used = row < count[:, None]
    at = (s["starts"][:-1, None] + row).long().clamp(max=s["tokens"] - 1)
    q = s["q"][at].float().unflatten(2, (h, g)).permute(0, 2, 3, 1, 4)  # [b, h, g, rows, d]
    score = torch.matmul(q.flatten(2, 3), k.transpose(2, 3).contiguous()).unflatten(2, (g, -1)) * s["scale"]
    p = (s["lens"] - count)[:, None] + row
    seen = (t <= p[..., None]) & (t < s["lens"][:, None, None])
    if case["window"]:
        seen &= (t > p[..., None] - case["window"]) | (t < case["sinks"])
    score = score.masked_fill_(~seen[:, None, None], -float("inf"))
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.flatten(2, 3), v).unflatten(2, (g, -1)) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[used].to(torch.bfloat16)


def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        nv = _lib()
        if kind == "quantize":
            return nv.mxfp4_dequantize(nv.mxfp4_quantize(s["x"]))
        if kind == "swiglu":
            return nv.mxfp4_dequantize(nv.mxfp4_quantize_swiglu(s["gate"], s["up"]))
        if kind == "gemm":
            return nv.mxfp4_gemm_bf16out(s["x"], s["w"])
        if kind == "linear":
            return nv.mxfp4_gemm_bf16out(nv.mxfp4_quantize(s["x"]), s["w"])
        if kind == "cache":
            nv.mxfp4_cache_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["starts"])
            return nv.mxfp4_cache_read(s["cache"], s["table"], s["lens"], s["starts"], s["tokens"])
        case = s["case"]
        return nv.mxfp4_attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"], scale=s["scale"],
                                  window=case["window"], sinks=case["sinks"], max_kv=s["longest"])
    if kind == "quantize":
        return _rounded(s["x"])
    if kind == "swiglu":
        return _rounded(_swiglu(s["gate"], s["up"]))
    if kind in ("gemm", "linear"):
        x = s["x"] if kind == "gemm" else _rounded(s["x"])
        return torch.matmul(x.float(), s["w"].float().t()).to(torch.bfloat16)
    if kind == "cache":
        _append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["starts"])
        return _read(s["cache"], s["table"], s["lens"], s["starts"], s["tokens"])
    return _attend(s)


# ---- the definition in 64 bits -------------------------------------------------------------

def _exact_two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_bf16(x):
    """float64 -> the nearest bf16 value, ties to even, as float64."""
    _, e = torch.frexp(x)
    e = e.clamp(min=-125)
    return torch.round(x * _exact_two(8 - e)) * _exact_two(e - 8)


def _exact_mx(x):
    """The MXFP4 value of each element, by search among the eight magnitudes, in float64."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 25) // max(1, x[0].numel()))
    for i in range(0, x.shape[0], step):  # rows at a time: the search holds several copies
        b = x[i:i + step].double().reshape(-1, BLOCK)
        top = b.abs().max(dim=1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        e = torch.where(_exact_two(e) > top, e - 1, torch.where(_exact_two(e + 1) <= top, e + 1, e))  # log2 is near
        scale = _exact_two(torch.where(top > 0, e - 2, -127.0).clamp(min=-127.0))
        y = (b.abs() / scale).clamp(max=6.0)
        low = (torch.searchsorted(values, y, right=True) - 1).clamp(max=6)
        down, up = y - values[low], values[low + 1] - y
        code = torch.where((up < down) | ((up == down) & (low % 2 == 1)), low + 1, low)
        out[i:i + step] = (torch.sign(b) * values[code] * scale).reshape(out[i:i + step].shape)
    return out


def _exact_product(a, w):
    out = torch.empty(a.shape[0], w.shape[0], dtype=torch.float64, device=a.device)
    for i in range(0, a.shape[0], 4096):
        out[i:i + 4096] = a[i:i + 4096] @ w.t()
    return out


def exact(case, seed):
    s, kind = _inputs(case, seed), case["kind"]
    if kind == "quantize":
        return _exact_mx(s["x"])
    if kind == "swiglu":
        y = torch.empty_like(s["gate"])
        for i in range(0, case["m"], 2048):
            g, u = s["gate"][i:i + 2048].double(), s["up"][i:i + 2048].double()
            y[i:i + 2048] = _exact_bf16(_exact_bf16(g * torch.sigmoid(g)) * u).to(torch.bfloat16)
        return _exact_mx(y)
    if kind in ("gemm", "linear"):
        return _exact_product(_exact_mx(s["x"]), _exact_mx(s["w"]))
    if kind == "cache":
        return _exact_mx(s["k"]), _exact_mx(s["v"])
    k, v, q = _exact_mx(s["k"]), _exact_mx(s["v"]), s["q"].double()
    new, cached = _lengths(case)
    out = torch.empty_like(q)
    g = case["heads"] // case["kv_heads"]
    q0 = k0 = 0
    for n, kv in zip(new, cached):
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        t = torch.arange(kv, device="cuda")[None]
        hidden = t > p
        if case["window"]:
            hidden |= (t <= p - case["window"]) & (t >= case["sinks"])
        for head in range(case["heads"]):
            a = q[q0:q0 + n, head] @ k[k0:k0 + kv, head // g].t() * case["dim"] ** -0.5
            a.masked_fill_(hidden, -float("inf"))
            out[q0:q0 + n, head] = torch.softmax(a, -1) @ v[k0:k0 + kv, head // g]
        q0, k0 = q0 + n, k0 + kv
    return out
