"""Workloads of what surrounds the MXFP4 cache: in plain torch, and through the library.

``run(state)`` is one pass. With ``own`` false it is the plain form: elementary torch
operations in fp32 (fp64 for angles, and for keys, whose 4-bit steps are cliffs), rounded
once at the end. With ``own`` true it is the calls a user of the library makes.

Kinds of case:

* ``rope``     norms and rotation of q and k by a position on each of several axes, bf16 out
* ``append``   the same for q; k and v go into their pages of an MXFP4 cache and are read back
* ``branch``   sequences continued in several ways: freed, forked, given pages, shared last pages copied
* ``compact``  used pages of a cache moved to its front
* ``prefix``   attention of sequences whose groups share their first pages
"""
import torch

own = False

BLOCK = 32
SPARE = 3  # pages of a cache that belong to no sequence


def _lib():
    import nvfp4_block_scaled_swiglu_amd as nv
    return nv


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one token of a long conversation on its way into the cache: launch latency
        {"name": "append_token", "kind": "append", "batch": 1, "q": 1, "kv": 131071, "heads": 32, "kv_heads": 4, "dim": 128,
         "page": 16, "rotary": 128, "axes": 1, "interleaved": False, "norm": True},
        # a decoding batch
        {"name": "append_batch", "kind": "append", "batch": 48, "q": 1, "kv": 8200, "heads": 56, "kv_heads": 8, "dim": 128,
         "page": 64, "rotary": 128, "axes": 1, "interleaved": False, "norm": True},
        # ragged prompts with images between their words, a quarter of the head turned
        {"name": "append_prompt", "kind": "append", "batch": 5, "q": 8191, "kv": 8191, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "rotary": 32, "axes": 3, "interleaved": False, "norm": True},
        # the video block's queries and keys: frame, row and column of each token
        {"name": "rope_video", "kind": "rope", "tokens": 37810, "heads": 56, "kv_heads": 56, "dim": 128, "rotary": 128,
         "axes": 3, "interleaved": True, "norm": True},
        # one prompt, 48 answers begin
        {"name": "branch_answers", "kind": "branch", "parents": 1, "children": 48, "prefix": 8200, "grow": 1, "kv_heads": 8,
         "dim": 128, "page": 64},
        # many prompts on small pages, 16 answers each, room for what comes next
        {"name": "branch_many", "kind": "branch", "parents": 64, "children": 16, "prefix": 8200, "grow": 37, "kv_heads": 8,
         "dim": 128, "page": 16},
        # a small cache after a few requests have left
        {"name": "compact_small", "kind": "compact", "groups": 4, "per": 4, "prefix": 500, "own": 200, "unused": 0.5,
         "kv_heads": 8, "dim": 128, "page": 64},
        # a large one, a third of it unused
        {"name": "compact_large", "kind": "compact", "groups": 32, "per": 8, "prefix": 8200, "own": 2000, "unused": 0.33,
         "kv_heads": 8, "dim": 128, "page": 64},
        # 48 answers to one prompt
        {"name": "prefix_answers", "kind": "prefix", "groups": 1, "per": 48, "prefix": 8200, "own": 500, "q": 1, "heads": 56,
         "kv_heads": 8, "dim": 128, "page": 64},
        # 16 answers to a very long one
        {"name": "prefix_long", "kind": "prefix", "groups": 1, "per": 16, "prefix": 131071, "own": 300, "q": 1, "heads": 32,
         "kv_heads": 4, "dim": 128, "page": 16},
        # a few answers to each of several prompts, drafted tokens checked, small heads
        {"name": "prefix_drafts", "kind": "prefix", "groups": 6, "per": 4, "prefix": 6000, "own": 700, "q": 5, "heads": 32,
         "kv_heads": 8, "dim": 64, "page": 32},
        # questions behind one set of instructions, read whole
        {"name": "prefix_questions", "kind": "prefix", "groups": 1, "per": 8, "prefix": 6200, "own": 512, "q": 512, "heads": 56,
         "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _log(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "branch", "compact", "prefix", "prefix", "prefix"])
    dim, kv_heads, page = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    if kind in ("rope", "append"):
        turn = {"dim": dim, "rotary": rng.choice([dim, dim, dim // 2, 32]), "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.7}
        if kind == "rope":
            return dict(turn, kind=kind, tokens=_log(rng, 1, 37810), heads=kv_heads * rng.choice([1, 3, 7]), kv_heads=kv_heads)
        q = rng.choice([1, _log(rng, 1, 8191)])
        return dict(turn, kind=kind, batch=_log(rng, 1, 48) if q < 512 else rng.randint(1, 5), q=q,
                    kv=_log(rng, q, 131071 if q < 512 else 8191), heads=kv_heads * rng.choice([1, 3, 4, 7]), kv_heads=kv_heads,
                    page=page)
    if kind == "branch":
        parents = _log(rng, 1, 64)
        return {"kind": kind, "parents": parents, "children": _log(rng, 1, max(1, 1024 // parents)), "prefix": _log(rng, 10, 8200),
                "grow": _log(rng, 1, 150), "kv_heads": kv_heads, "dim": dim, "page": page}
    if kind == "compact":
        return {"kind": kind, "groups": _log(rng, 1, 32), "per": _log(rng, 1, 8), "prefix": _log(rng, 10, 8200),
                "own": _log(rng, 5, 2000), "unused": 0.1 + 0.8 * rng.random(), "kv_heads": kv_heads, "dim": dim, "page": page}
    heads = kv_heads * rng.choice([1, 3, 4, 7])
    form = rng.choice(["answers", "answers", "long", "questions"])
    if form == "answers":
        groups, per, prefix, at, q = _log(rng, 1, 6), _log(rng, 2, 8), _log(rng, 64, 8200), _log(rng, 5, 700), rng.choice([1, 1, 3, 5])
    elif form == "long":
        groups, per, prefix, at, q = 1, _log(rng, 2, 16), _log(rng, 8192, 131071), _log(rng, 1, 300), 1
    else:
        groups, per, prefix, at = 1, _log(rng, 2, 8), _log(rng, 64, 6200), _log(rng, 16, 512)
        q = at
    return {"kind": kind, "groups": groups, "per": per, "prefix": prefix, "own": at, "q": q, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page}


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: ragged, the first the longest."""
    b = case["batch"]
    kv = [max(1, case["kv"] - i * (case["kv"] // (2 * b))) for i in range(b)]
    q = [min(kv[i], max(1, case["q"] - i * (case["q"] // (3 * b)))) for i in range(b)]
    return q, kv


def _family(groups, per, prefix, own_tokens):
    """(prefix of each group, own tokens of each sequence): ragged, the first the longest."""
    n = groups * per
    return ([max(1, prefix - g * (prefix // (2 * groups))) for g in range(groups)],
            [max(1, own_tokens - i * (own_tokens // (2 * n))) for i in range(n)])


def _page_bytes(case):
    return 2 * case["kv_heads"] * case["page"] * (case["dim"] // 2 + case["dim"] // BLOCK)


def work(case):
    kind = case["kind"]
    packed = 0.5 + 1 / BLOCK  # bytes of an MXFP4 element with its share of a scale
    if kind == "rope":
        e = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * e, "flops": 8 * e}
    if kind == "append":
        t = sum(_lengths(case)[0]) * case["dim"]
        return {"bytes": t * (case["heads"] * 4 + 2 * case["kv_heads"] * (2 + packed + packed + 2)),
                "flops": 8 * t * (case["heads"] + 2 * case["kv_heads"])}
    if kind == "branch":
        pages = -(-(case["prefix"] + 1) // case["page"])
        n = case["parents"] * case["children"]
        return {"bytes": 4 * (case["parents"] * pages + n * pages) + n * 2 * _page_bytes(case), "flops": 0}
    if kind == "compact":
        shared, own_tokens = _family(case["groups"], case["per"], case["prefix"], case["own"])
        page = case["page"]
        used = sum(n // page for n in shared) + sum(-(-(shared[i // case["per"]] + n) // page) - shared[i // case["per"]] // page
                                                    for i, n in enumerate(own_tokens))
        table = sum(-(-(shared[i // case["per"]] + n) // page) for i, n in enumerate(own_tokens))
        count = used + int(used * case["unused"] / (1 - case["unused"])) + SPARE
        moved = used * (count - used) // count  # of pages in random places
        return {"bytes": 8 * (count + table) + moved * 2 * _page_bytes(case), "flops": 0}
    shared, own_tokens = _family(case["groups"], case["per"], case["prefix"], case["own"])
    rows = [min(n, case["q"]) for n in own_tokens]
    pairs = sum(r * (shared[i // case["per"]] + n) - r * (r - 1) // 2 for i, (r, n) in enumerate(zip(rows, own_tokens)))
    return {"bytes": 2 * (sum(shared) + sum(own_tokens)) * case["kv_heads"] * case["dim"] * packed
            + 4 * sum(rows) * case["heads"] * case["dim"], "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---- inputs --------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, seed, sigma=1.0, outliers=False):
    """bf16 N(0, sigma); with outliers every 100th channel is 20 times as large, as in the block's activations."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, sigma, generator=_generator(seed))
    if outliers:
        x[..., 7::100] *= 20
    return x


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    return _ints([0] + counts).cumsum(0).to(torch.int32)


def _pages_of(case, groups, per, prefix, own_tokens, seed, unused=0.0, more=0):
    """Sequences whose groups share the full pages of their prefix, their pages in random places:
    block table, lengths, prefix lengths in whole pages, entries that hold each page."""
    page = case["page"]
    shared, own_tokens = _family(groups, per, prefix, own_tokens)
    full = [n // page for n in shared]
    lens = [shared[i // per] + n for i, n in enumerate(own_tokens)]
    held = [-(-n // page) for n in lens]
    used = sum(full) + sum(h - full[i // per] for i, h in enumerate(held))
    count = used + int(used * unused / (1 - unused)) + SPARE + more
    order = torch.randperm(count, generator=_generator(seed + 11), device="cuda").to(torch.int32)
    most = max(held) + -(-case.get("grow", 0) // page)
    e = torch.arange(most, device="cuda")
    group = torch.arange(groups * per, device="cuda") // per
    f, h = _ints(full)[group][:, None], _ints(held)[:, None]
    first = _starts(full)[group][:, None] + e
    rest = sum(full) + _starts([n - full[i // per] for i, n in enumerate(held)])[:-1][:, None] + e - f
    at = torch.where(e < f, first, rest).clamp(0, count - 1).long()
    table = torch.where(e < h, order[at], -1).to(torch.int32)
    refs = torch.zeros(count, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, table.clamp(min=0).long().flatten(), (table >= 0).int().flatten())
    return table, _ints(lens), _ints(full) * page, refs


def _filled(case, count, seed):
    """A cache full of quantized keys and values: codes and scales of both."""
    shape = (count, case["kv_heads"], case["page"], case["dim"])
    kv = []
    for i in range(2):
        codes = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device="cuda")
        scales = torch.empty(shape[:-1] + (shape[-1] // BLOCK,), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
        for p in range(0, count, step):
            x = _normal((min(step, count - p),) + shape[1:], seed + 2 * p + i, outliers=i == 0)
            codes[p:p + step], scales[p:p + step] = _encode(x)
        kv += [codes, scales]
    return kv


def _turns(case, tokens, seed, positions=None):
    """What turns the heads: frequencies of the pairs, their axes, positions; and the norms' weights."""
    n = case["rotary"] // 2
    each = [n // case["axes"] + (a < n % case["axes"]) for a in range(case["axes"])]
    s = {"axes": _ints([a for a, c in enumerate(each) for _ in range(c)]),
         "freqs": torch.tensor([10000.0 ** (-i / c) for c in each for i in range(c)], dtype=torch.float32, device="cuda")}
    if case["axes"] > 1:  # frame, row and column of a sweep over a clip (the words of a prompt go the same way)
        t = torch.arange(tokens, dtype=torch.int32, device="cuda")
        s["positions"] = torch.stack([t // 1200, t // 40 % 30, t % 40], 1)[:, :case["axes"]].contiguous()
    else:
        s["positions"] = None if positions is None else positions
    if case["norm"]:
        s["qw"], s["kw"] = (1 + _normal((case["dim"],), seed + i, 0.1) for i in (5, 6))
    return s


def _inputs(case, seed):
    """What a program has in hand before the call, from the seed alone."""
    kind = case["kind"]
    if kind == "rope":
        t, d = case["tokens"], case["dim"]
        return dict(_turns(case, t, seed, torch.arange(t, dtype=torch.int32, device="cuda")),
                    q=_normal((t, case["heads"], d), seed, 2.0), k=_normal((t, case["kv_heads"], d), seed + 1, 2.0, True))
    if kind == "append":
        q, kv = _lengths(case)
        page = case["page"]
        held = [-(-n // page) for n in kv]
        count = sum(held) + SPARE
        order = torch.randperm(count, generator=_generator(seed + 11), device="cuda").to(torch.int32)
        e = torch.arange(max(held), device="cuda")
        at = (_starts(held)[:-1][:, None] + e).clamp(max=count - 1).long()
        new, h, d = sum(q), case["kv_heads"], case["dim"]
        s = _turns(case, new, seed)
        qkv = _normal((new, case["heads"] + 2 * h, d), seed, 2.0)  # as the projection leaves them
        qkv[:, case["heads"]:-h, 7::100] *= 20
        s.update(q=qkv[:, :case["heads"]], k=qkv[:, case["heads"]:-h], v=qkv[:, -h:], lens=_ints(kv), starts=_starts(q),
                 table=torch.where(e < _ints(held)[:, None], order[at], -1).to(torch.int32), new=new)
        shape = (count, h, page)
        s["cache"] = [torch.zeros(shape + (n,), dtype=torch.uint8, device="cuda") for n in (d // 2, d // BLOCK) * 2]
        return s
    if kind == "branch":
        p, c = case["parents"], case["children"]
        need = p * c * (1 + -(-case["grow"] // case["page"]))
        table, lens, _, refs = _pages_of(case, p, 1, case["prefix"], 1, seed, more=need)
        s = {"table": torch.cat([table, torch.full((p * c, table.shape[1]), -1, dtype=torch.int32, device="cuda")]),
             "lens": torch.cat([lens, torch.zeros(p * c, dtype=torch.int32, device="cuda")]), "refs": refs,
             "parents": torch.arange(p, device="cuda").repeat_interleave(c).to(torch.int32),
             "children": torch.arange(p, p + p * c, device="cuda").to(torch.int32)}
        s["grown"] = s["lens"][s["parents"].long()] + case["grow"]
        return dict(s, cache=_bytes(case, refs.shape[0], seed))
    table, lens, shared, refs = _pages_of(case, case["groups"], case["per"], case["prefix"], case["own"], seed,
                                          unused=case.get("unused", 0.0))
    s = {"table": table, "lens": lens, "refs": refs}
    if kind == "compact":
        return dict(s, cache=_bytes(case, refs.shape[0], seed))
    own_tokens = _family(case["groups"], case["per"], case["prefix"], case["own"])[1]
    rows = [min(n, case["q"]) for n in own_tokens]
    return dict(s, cache=_filled(case, refs.shape[0], seed), starts=_starts(rows), most=max(rows), longest=max(own_tokens) + case["page"],
                q=_normal((sum(rows), case["heads"], case["dim"]), seed + 2), prefix_table=table[::case["per"]].contiguous(),
                prefix_lens=shared, groups=_starts([case["per"]] * case["groups"]), scale=case["dim"] ** -0.5)


def _bytes(case, count, seed):
    """A cache whose contents are only moved: any bytes."""
    shape, d = (count, case["kv_heads"], case["page"]), case["dim"]
    return [torch.randint(0, 256, shape + (n,), dtype=torch.uint8, device="cuda", generator=_generator(seed + 20 + i))
            for i, n in enumerate((d // 2, d // BLOCK) * 2)]


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# ---- the plain form ------------------------------------------------------------------------

def _two(e):
    """2^e in fp32 for whole -127 <= e <= 127, by its bits (a power function may be an ulp off)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _encode(x):
    """bf16 [..., d] -> MXFP4 codes [..., d / 2] and scales [..., d / 32]."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(min=-127)
    a = b.abs() * _two(-e)
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = (c + 8 * torch.signbit(b)).flatten(-2).to(torch.uint8)
    return c[..., ::2] | (c[..., 1::2] << 4), (e + 127).squeeze(-1).to(torch.uint8)


def _decode(codes, scales):
    """The values, in fp32."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    m = c & 7
    v = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8))
    v = torch.where(c > 7, -v, v).unflatten(-1, (-1, BLOCK))
    return (v * _two(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _nearest(x):
    """RN_bf16 of fp64 values, their rounding to fp32 on the way kept off the ties."""
    f = x.float()
    bits = f.view(torch.int32)
    tie = (bits & 0xFFFF) == 0x8000
    off = (x.abs() > f.double().abs()).int() - (x.abs() < f.double().abs()).int()
    return (bits + tie * off).view(torch.float32).to(torch.bfloat16)


def _turned(x, s, weight, positions, dtype):
    """Norm and rotation of [tokens, heads, dim] in `dtype`; angles in fp64."""
    case = s["case"]
    y = x.to(dtype)
    if case["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s[weight].to(dtype)
    if positions.dim() == 1:
        positions = positions[:, None]
    angle = positions.double()[:, s["axes"].long()] * s["freqs"].double()
    cos, sin = torch.cos(angle).to(dtype)[:, None], torch.sin(angle).to(dtype)[:, None]
    r = case["rotary"]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    a, b = a * cos - b * sin, b * cos + a * sin
    t = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([t, y[..., r:]], -1)


def _places(s):
    """(page, slot in it, position) of each new token: the last ones of its sequence."""
    row = torch.arange(s["new"], device="cuda")
    seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    at = s["lens"][seq].long() - s["starts"][seq + 1] + row
    page = s["case"]["page"]
    return s["table"][seq, at // page].long(), at % page, at


def _append(s):
    page, slot, at = _places(s)
    at = at if s["positions"] is None else s["positions"]
    for i, x in enumerate((_nearest(_turned(s["k"], s, "kw", at, torch.float64)), s["v"])):
        s["cache"][2 * i][page, :, slot], s["cache"][2 * i + 1][page, :, slot] = _encode(x)
    q = _turned(s["q"], s, "qw", at, torch.float32).to(torch.bfloat16)
    return (q,) + tuple(_decode(s["cache"][i][page, :, slot], s["cache"][i + 1][page, :, slot]).to(torch.bfloat16) for i in (0, 2))


def _holds(lens, page):
    return (lens + page - 1) // page


def _branch(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    child, parent = s["children"].long(), s["parents"].long()
    e = torch.arange(table.shape[1], device="cuda")

    def count(rows, held, by):
        mask = e < held[:, None]
        refs.scatter_add_(0, torch.where(mask, rows, 0).long().flatten(), (by * mask).int().flatten())
        return mask

    # free
    gone = count(table[child], _holds(lens[child], page), -1)
    table[child] = torch.where(gone, -1, table[child])
    lens[child] = 0
    # fork
    kept = count(table[parent], _holds(lens[parent], page), 1)
    table[child] = torch.where(kept, table[parent], table[child])
    lens[child] = lens[parent]
    # reserve: the lowest free pages, in the order of the list; a shared last page is copied before it is written
    old, new = lens[child], s["grown"]
    have, want = _holds(old, page), _holds(new, page)
    last = table[child, (have - 1).clamp(min=0).long()]
    copied = (old % page > 0) & (new > old) & (refs[last.clamp(min=0).long()] > 1)
    need = torch.where(new >= old, want - have + copied.int(), 0)
    upto = need.cumsum(0)
    done = (new >= old) & (want <= e.numel()) & (upto <= (refs == 0).sum())
    copied &= done
    free = torch.argsort((refs != 0).int(), stable=True).to(torch.int32)
    number = (upto - need)[:, None] + torch.where(e < have[:, None], 0, copied.int()[:, None] + e - have[:, None])
    fresh = done[:, None] & (((e >= have[:, None]) & (e < want[:, None])) | (copied[:, None] & (e == have[:, None] - 1)))
    pages = torch.where(fresh, free[number.clamp(0, free.numel() - 1).long()], 0)
    src, dst = torch.where(copied, last, -1), torch.where(copied, free[(upto - need).clamp(max=free.numel() - 1).long()], -1)
    refs.scatter_add_(0, pages.long().flatten(), fresh.int().flatten())
    refs.scatter_add_(0, src.clamp(min=0).long(), -copied.int())
    table[child] = torch.where(fresh, pages, table[child])
    lens[child] = torch.where(done, new, old)
    _copy(s["cache"], src, dst)
    return [table, lens, refs, done.int(), src, dst] + s["cache"]


def _copy(cache, src, dst):
    """Pages src -> dst; a pair of -1 moves nothing (page dst's own contents to itself)."""
    live = src >= 0
    spare = torch.argmax(live.int())  # a pair that is there, if any is
    to = torch.where(live, dst, dst[spare]).clamp(min=0).long()
    at = torch.where(live, src, src[spare])
    at = torch.where(at >= 0, at, 0).long()
    for c in cache:
        c[to] = c[at]


def _compact(s):
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    n = refs.shape[0]
    used = (refs > 0).sum()
    at = torch.arange(n, device="cuda")
    leaves, hole = (at >= used) & (refs > 0), (at < used) & (refs <= 0)
    src = torch.argsort((~leaves).int(), stable=True)[:n // 2]
    dst = torch.argsort((~hole).int(), stable=True)[:n // 2]
    live = torch.arange(n // 2, device="cuda") < leaves.sum()
    to = at.clone()
    to[torch.where(live, src, n - 1)] = torch.where(live, dst, to[n - 1])  # (the last page, if it moves at all, is the last mover)
    last = torch.where(leaves[n - 1], dst[(leaves.sum() - 1).clamp(0, n // 2 - 1)], n - 1)
    to[n - 1] = last
    mask = torch.arange(table.shape[1], device="cuda") < _holds(s["lens"], page)[:, None]
    moved = torch.where(mask, to[table.clamp(min=0).long()].to(torch.int32), table)
    counts = torch.zeros_like(refs).scatter_add_(0, to, refs * (refs > 0))
    src, dst = (torch.where(live, x, -1).to(torch.int32) for x in (src, dst))
    _copy(s["cache"], src, dst)
    return [moved, counts, src, dst, used.to(torch.int32).reshape(1)] + s["cache"]


def _attend(s):
    case = s["case"]
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    g = case["heads"] // h
    table = s["table"].long().clamp(min=0)
    k, v = (_decode(s["cache"][i][table], s["cache"][i + 1][table]).transpose(1, 2).flatten(2, 3) for i in (0, 2))
    t = torch.arange(k.shape[2], device="cuda")
    count = s["starts"][1:] - s["starts"][:-1]
    row = torch.arange(s["most"], device="cuda")
    used = row < count[:, None]
    at = (s["starts"][:-1, None] + row).long().clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().unflatten(2, (h, g)).permute(0, 2, 3, 1, 4)  # [b, h, g, rows, d]
    score = torch.matmul(q.flatten(2, 3), k.transpose(2, 3).contiguous()).unflatten(2, (g, -1)) * s["scale"]
    seen = t <= ((s["lens"] - count)[:, None] + row)[..., None]
    score = score.masked_fill_(~seen[:, None, None], -float("inf"))
    score = score.sub_(score.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(score.flatten(2, 3), v).unflatten(2, (g, -1)) / score.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[used].to(torch.bfloat16)


def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        nv = _lib()
        case = s["case"]
        if kind in ("rope", "append"):
            turn = nv.Mxfp4Rotation(s["freqs"], s["axes"], case["axes"], case["interleaved"])
            eps = 1e-6 if case["norm"] else None
            if kind == "rope":
                return [nv.mxfp4_norm_rope(s[n], turn, s["positions"], weight=s.get(n + "w"), eps=eps) for n in ("q", "k")]
            cache = nv.Mxfp4Cache(*s["cache"])
            q = nv.mxfp4_norm_rope_append(cache, s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], turn, s["positions"],
                                          q_weight=s.get("qw"), k_weight=s.get("kw"), eps=eps)
            return (q,) + nv.mxfp4_cache_read(cache, s["table"], s["lens"], s["starts"], s["new"])
        cache = nv.Mxfp4Cache(*s["cache"])
        if kind == "prefix":
            return nv.mxfp4_attention_prefix(s["q"], cache, s["table"], s["lens"], s["starts"], s["prefix_table"],
                                             s["prefix_lens"], s["groups"], scale=s["scale"], max_own=s["longest"],
                                             max_prefix=case["prefix"])
        pages = nv.Mxfp4Pages(s["table"], s["lens"], s["refs"], case["page"])
        if kind == "branch":
            nv.mxfp4_pages_free(pages, s["children"])
            nv.mxfp4_pages_fork(pages, s["parents"], s["children"])
            done, src, dst = nv.mxfp4_pages_reserve(pages, s["children"], s["grown"])
            nv.mxfp4_cache_copy(cache, src, dst)
            return [s["table"], s["lens"], s["refs"], done, src, dst] + s["cache"]
        after, src, dst, used = nv.mxfp4_pages_compact(pages)
        nv.mxfp4_cache_copy(cache, src, dst)
        return [after.block_table, after.refs, src, dst, used] + s["cache"]
    if kind == "rope":
        return [_turned(s[n], s, n + "w", s["positions"], torch.float32).to(torch.bfloat16) for n in ("q", "k")]
    if kind == "append":
        return _append(s)
    return {"branch": _branch, "compact": _compact, "prefix": _attend}[kind](s)


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
    b = x.double().reshape(-1, BLOCK)
    top = b.abs().max(dim=1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(_exact_two(e) > top, e - 1, torch.where(_exact_two(e + 1) <= top, e + 1, e))  # log2 is near
    scale = _exact_two(torch.where(top > 0, e - 2, -127.0).clamp(min=-127.0))
    y = (b.abs() / scale).clamp(max=6.0)
    low = (torch.searchsorted(values, y, right=True) - 1).clamp(max=6)
    down, up = y - values[low], values[low + 1] - y
    code = torch.where((up < down) | ((up == down) & (low % 2 == 1)), low + 1, low)
    return (torch.sign(b) * values[code] * scale).reshape(x.shape)


def _exact_turned(x, s, case, weight, positions):
    """Pair by pair, as complex numbers turned by e^(i angle)."""
    y = x.double()
    if case["norm"]:
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / case["dim"] + 1e-6) * s[weight].double()
    r = case["rotary"]
    out = y.clone()
    for j in range(r // 2):
        i, k = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + r // 2)
        p = positions if positions.dim() == 1 else positions[:, int(s["axes"][j])]
        angle = (p.double() * float(s["freqs"][j]))[:, None]
        z = torch.complex(y[..., i], y[..., k]) * torch.polar(torch.ones_like(angle), angle)
        out[..., i], out[..., k] = z.real, z.imag
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind in ("branch", "compact"):
        return None  # whole numbers and bytes that move
    s = _inputs(case, seed)
    if kind == "rope":
        return [_exact_turned(s[n], s, case, n + "w", s["positions"]) for n in ("q", "k")]
    if kind == "append":
        q, kv = _lengths(case)
        at = s["positions"]
        if at is None:
            at = torch.cat([torch.arange(n - c, n, device="cuda") for c, n in zip(q, kv)])
        return (_exact_turned(s["q"], s, case, "qw", at), _exact_mx(_exact_bf16(_exact_turned(s["k"], s, case, "kw", at))),
                _exact_mx(s["v"]))
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    values = torch.cat([values, -values])
    q, g, page = s["q"].double(), case["heads"] // case["kv_heads"], case["page"]
    out = torch.empty_like(q)
    starts = s["starts"].tolist()
    for i, n in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :-(-n // page)].long()
        kv = []
        for codes, scales in (s["cache"][:2], s["cache"][2:]):
            c, e = codes[pages].transpose(1, 2).flatten(0, 1)[:n].long(), scales[pages].transpose(1, 2).flatten(0, 1)[:n]
            x = torch.stack([values[c % 16], values[c // 16]], -1).flatten(-2)
            kv.append(x * _exact_two(e.long() - 127).repeat_interleave(BLOCK, -1))
        rows = slice(starts[i], starts[i + 1])
        p = torch.arange(n - (starts[i + 1] - starts[i]), n, device="cuda")[:, None]
        hidden = torch.arange(n, device="cuda")[None] > p
        for head in range(case["heads"]):
            a = q[rows, head] @ kv[0][:, head // g].t() * case["dim"] ** -0.5
            out[rows, head] = torch.softmax(a.masked_fill_(hidden, -float("inf")), -1) @ kv[1][:, head // g]
    return out
