"""Host-side checks of the operators around the MXFP4 cache (no GPU): every refusal returns its status
before a device is touched, limits are where the header says, and the binding refuses what does not fit."""
import ctypes

import pytest

import nvfp4_block_scaled_swiglu_amd as nv
from nvfp4_block_scaled_swiglu_amd import mxfp4
from tests.test_mx_host import CACHE, CACHE_REFUSALS, FAKE, structs

NO_DEVICE = 5


def passed(status):
    """What a call that passes the validation returns here; with a GPU it must not be made."""
    import torch
    if status == 0 and torch.cuda.is_available():
        pytest.skip("a GPU is visible: a call that passes would run")
    return NO_DEVICE if status == 0 else status


NORM = dict(weight=FAKE, eps=1e-6)
ROT = dict(freqs=FAKE, axes_dev=FAKE, positions=FAKE, rotary=32, axes=3, pt=3, pa=1, inter=0)
ROPE = dict(x=FAKE, xt=256, xh=64, tokens=8, heads=4, dim=64, norm=1, rot=1, out=FAKE, ot=256, oh=64, st=None)

ROTATIONS = [
    ({}, 0), (dict(freqs=None), 1), (dict(freqs=FAKE + 2), 3), (dict(axes_dev=None), 0), (dict(axes_dev=FAKE + 1), 3),
    (dict(positions=FAKE + 2), 3), (dict(rotary=0), 1), (dict(rotary=-16), 1), (dict(rotary=8), 2), (dict(rotary=80), 1),
    (dict(rotary=64), 0), (dict(rotary=40), 2), (dict(axes=0), 1), (dict(axes=64), 0), (dict(axes=65), 2), (dict(pt=-1), 1),
    (dict(pa=-1), 1), (dict(pt=1 << 31, pa=1 << 31), 0), (dict(pt=(1 << 31) + 1), 2), (dict(pa=(1 << 31) + 1), 2), (dict(pt=0), 0),
]
NORMS = [(dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(eps=1e-300), 0),
         (dict(weight=None), 0), (dict(weight=FAKE + 8), 3)]


def turns(kw):
    return (mxfp4._CNorm(*{**NORM, **{n: v for n, v in kw.items() if n in NORM}}.values()),
            mxfp4._CRotation(*{**ROT, **{n: v for n, v in kw.items() if n in ROT}}.values()))


def rope(kw):
    norm, rot = turns(kw)
    a = {**ROPE, **{n: v for n, v in kw.items() if n in ROPE}}
    a["norm"], a["rot"] = norm if a["norm"] else None, rot if a["rot"] else None
    return nv.lib().mxfp4_norm_rope(*a.values())


@pytest.mark.parametrize("kw,status", ROTATIONS + NORMS + [
    (dict(norm=0, rot=0), 0), (dict(norm=0), 0), (dict(rot=0), 0), (dict(positions=None), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(heads=65537, xt=1 << 23, ot=1 << 23), 2), (dict(dim=96), 2), (dict(dim=0), 1),
    (dict(x=FAKE + 8), 3), (dict(xh=60), 3), (dict(ot=250), 3), (dict(oh=0), 1), (dict(ot=64), 1), (dict(xt=-8), 1), (dict(xt=0, xh=0), 0),
    (dict(xt=(1 << 31) + 8), 2), (dict(tokens=(1 << 26) - 4), 0), (dict(tokens=(1 << 26) - 3), 2), (dict(heads=65536, ot=1 << 22), 0),
    (dict(tokens=0, x=None, out=None, positions=None), 0),
])
def test_norm_rope(kw, status):
    want = passed(status)
    assert rope(kw) == want
    assert want == 0 or nv.lib().nvfp4_last_error().decode() != ""


APPEND = dict(q=FAKE, qt=512, qh=64, heads=4, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, out=FAKE, ot=256, oh=64)


def append(kw):
    c, b = structs(kw)
    norm, rot = turns(kw)
    a = {**APPEND, **{n: v for n, v in kw.items() if n in APPEND}}
    return nv.lib().mxfp4_norm_rope_append(
        c, b, a["q"], a["qt"], a["qh"], a["heads"], norm if kw.get("qn", 1) else None, a["k"], a["kt"], a["kh"],
        norm if kw.get("kn", 1) else None, a["v"], a["vt"], a["vh"], rot if kw.get("rot", 1) else None, a["out"], a["ot"], a["oh"], None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + ROTATIONS + NORMS + [
    (dict(qn=0, kn=0, rot=0), 0), (dict(positions=None), 0), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1),
    (dict(heads=-1), 1), (dict(heads=0, q=None, out=None), 0), (dict(heads=65537), 2), (dict(heads=3), 0), (dict(k=FAKE + 2), 3),
    (dict(vh=60), 3), (dict(kt=1 << 32), 2), (dict(ot=64), 1), (dict(out=FAKE + 8), 3), (dict(b_tokens=(1 << 26) - 4), 0),
    (dict(b_tokens=(1 << 26) - 3), 2), (dict(b_tokens=0, q=None, k=None, v=None, out=None), 0),
    (dict(b_batch=0, q=None, k=None, v=None, out=None), 0),
])
def test_append(kw, status):
    assert append(kw) == passed(status)


PREFIX = dict(table=FAKE, lens=FAKE, starts=FAKE, groups=2, pages=2, stride=2)
ATTN = dict(q=FAKE, qt=256, qh=64, heads=4, scale=0.125, causal=1, mp=32, mo=32, out=FAKE, ot=256, oh=64, ws=FAKE, wb=1 << 40, st=None)


def prefix(kw):
    c, b = structs(kw)
    x = mxfp4._CPrefix(*{**PREFIX, **{n[2:]: v for n, v in kw.items() if n.startswith("x_")}}.values())
    a = {**ATTN, **{n: v for n, v in kw.items() if n in ATTN}}
    return nv.lib().mxfp4_attention_prefix(c, b, x, *a.values()), nv.lib().mxfp4_attention_prefix_workspace_bytes(
        c, b, x, a["heads"], a["mp"], a["mo"])


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    ({}, 0), (dict(x_table=None), 1), (dict(x_lens=None), 1), (dict(x_starts=None), 1), (dict(x_starts=FAKE + 2), 3),
    (dict(x_table=None, x_pages=0, x_stride=0), 0), (dict(x_groups=-1), 1), (dict(x_groups=0), 0), (dict(x_stride=1), 1),
    (dict(x_pages=-1), 1), (dict(x_groups=1 << 24), 2), (dict(x_pages=1 << 26, x_stride=1 << 26), 2), (dict(mp=0), 1), (dict(mo=0), 1),
    (dict(heads=3), 1), (dict(heads=0), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(scale=2.0 ** 127), 0),
    (dict(q=None), 1), (dict(out=None), 1), (dict(qh=60), 3), (dict(ot=64), 1), (dict(ws=None), 4), (dict(wb=64), 4), (dict(ws=FAKE + 4), 3),
    (dict(b_tokens=(1 << 24) - 1), 0), (dict(b_tokens=1 << 24), 2), (dict(x_groups=(1 << 23) - 5, x_stride=2), 0),
    (dict(x_groups=(1 << 23) - 4, x_stride=2), 2), (dict(x_groups=1 << 22, b_batch=(1 << 22) - 3), 0), (dict(x_groups=1 << 22, b_batch=(1 << 22) - 2), 2), (dict(b_tokens=0, q=None, out=None, ws=None, wb=0, x_table=None), 0),
])
def test_attention_prefix(kw, status):
    want = passed(status)
    rc, size = prefix(kw)
    assert rc == want
    sizes_fine = {"q", "out", "qh", "ot", "ws", "wb", "scale"}
    if want == NO_DEVICE or set(kw) <= sizes_fine:
        assert size >= 0
    else:
        assert size == -1 or "null" in nv.lib().nvfp4_last_error().decode()


def test_prefix_workspace():
    """Two pieces at least of 64 + 2 floats a row and head, and a word a row; none without rows; that of mxfp4_attention without groups."""
    assert prefix({})[1] == 2 * 8 * 4 * 66 * 4 + 8 * 4
    assert prefix(dict(b_tokens=0))[1] == 0
    assert prefix(dict(mp=1 << 17))[1] > prefix({})[1]
    # groups without rows take a share of the launch: with very many of them there are no further pieces
    assert prefix(dict(mp=1 << 17, x_groups=1 << 16))[1] == prefix({})[1]
    c, b = structs({})
    x = mxfp4._CPrefix(None, None, None, 0, 0, 0)
    assert nv.lib().mxfp4_attention_prefix_workspace_bytes(c, b, x, 4, 1, 1 << 17) == \
        nv.lib().mxfp4_attention_workspace_bytes(c, b, 4, 1 << 17, 0, 0) > 0


PAGES = dict(table=FAKE, lens=FAKE, refs=FAKE, slots=4, most=6, stride=6, num=50, size=16)
PAGES_REFUSALS = [
    (dict(table=None), 1), (dict(lens=None), 1), (dict(refs=None), 1), (dict(refs=FAKE + 2), 3), (dict(slots=0), 1), (dict(most=0), 1),
    (dict(num=0), 1), (dict(stride=5), 1), (dict(size=24), 2), (dict(size=8), 2), (dict(size=65536), 2), (dict(slots=1 << 24), 2),
    (dict(num=1 << 31), 2), (dict(most=1 << 26, stride=1 << 26), 2), (dict(stride=1 << 41), 2),
]
LISTS = [(dict(n=-1), 1), (dict(n=65536), 2), (dict(n=65535), 0), (dict(a=None), 1), (dict(a=FAKE + 2), 3), (dict(n=0, a=None, b=None, d=None), 0)]


def pages_of(kw):
    return mxfp4._CPages(*{**PAGES, **{n: v for n, v in kw.items() if n in PAGES}}.values())


def lists(kw):
    return {**dict(a=FAKE, b=FAKE, n=3, d=FAKE, s=FAKE, t=FAKE, ws=FAKE, wb=1 << 40), **kw}


@pytest.mark.parametrize("kw,status", PAGES_REFUSALS + LISTS + [(dict(b=None), 0), (dict(b=FAKE + 1), 3), ({}, 0)])
def test_free(kw, status):
    a = lists(kw)
    assert nv.lib().mxfp4_pages_free(pages_of(kw), a["a"], a["b"], a["n"], None) == passed(status)


@pytest.mark.parametrize("kw,status", PAGES_REFUSALS + LISTS + [(dict(b=None), 1), (dict(d=None), 1), (dict(d=FAKE + 1), 3), ({}, 0)])
def test_fork(kw, status):
    a = lists(kw)
    assert nv.lib().mxfp4_pages_fork(pages_of(kw), a["a"], a["b"], a["n"], a["d"], None) == passed(status)


@pytest.mark.parametrize("kw,status", PAGES_REFUSALS + LISTS + [
    (dict(b=None), 1), (dict(d=None), 1), (dict(s=None), 1), (dict(t=FAKE + 2), 3), (dict(ws=None), 4), (dict(wb=63), 4), (dict(ws=FAKE + 8), 3),
    ({}, 0),
])
def test_reserve(kw, status):
    a, p = lists(kw), pages_of(kw)
    assert nv.lib().mxfp4_pages_reserve(p, a["a"], a["b"], a["n"], a["d"], a["s"], a["t"], a["ws"], a["wb"], None) == passed(status)
    size = nv.lib().mxfp4_pages_reserve_workspace_bytes(p, a["n"])
    assert (size == -1) == ((kw, status) in PAGES_REFUSALS or a["n"] in (-1, 65536))


@pytest.mark.parametrize("kw,status", PAGES_REFUSALS + [
    (dict(out=None), 1), (dict(ostride=5), 1), (dict(ostride=(1 << 40) + 1), 1), (dict(out=FAKE, ostride=7), 1), (dict(orefs=None), 1),
    (dict(s=None), 1), (dict(t=FAKE + 2), 3), (dict(d=None), 1), (dict(ws=None), 4), (dict(wb=8), 4), (dict(ws=FAKE + 4), 3), ({}, 0),
    (dict(num=1, s=None, t=None), 0), (dict(slots=(1 << 24) - 2), 0), (dict(slots=(1 << 24) - 1), 2), (dict(slots=1 << 23, most=257, stride=257, ostride=257), 2),
])
def test_compact(kw, status):
    a = {**dict(out=2 * FAKE, ostride=6, orefs=FAKE), **lists(kw)}
    p = pages_of(kw)
    rc = nv.lib().mxfp4_pages_compact(p, a["out"], a["ostride"], a["orefs"], a["s"], a["t"], a["d"], a["ws"], a["wb"], None)
    assert rc == passed(status)


@pytest.mark.parametrize("kw,status", [(dict(CACHE_REFUSALS[i][0]), CACHE_REFUSALS[i][1]) for i in range(11)] + [
    ({}, 0), (dict(a=None), 1), (dict(b=FAKE + 2), 3), (dict(n=-1), 1), (dict(n=1 << 31), 2), (dict(n=(1 << 31) - 1), 0), (dict(n=0, a=None, b=None), 0),
    (dict(o_size=32), 1), (dict(o_heads=3), 1), (dict(o_dim=128), 1), (dict(o_pages=9), 0), (dict(o_vc=None), 1),
])
def test_copy(kw, status):
    c, _ = structs(kw)
    to = mxfp4._CCache(*{**CACHE, **{n[2:]: v for n, v in kw.items() if n.startswith("o_")}}.values())
    a = lists(kw)
    assert nv.lib().mxfp4_cache_copy(c, to, a["a"], a["b"], a["n"], None) == passed(status)


def test_null_records():
    c, b = structs({})
    l = nv.lib()
    assert l.mxfp4_pages_free(None, FAKE, None, 1, None) == 1 == l.mxfp4_pages_fork(None, FAKE, FAKE, 1, FAKE, None)
    assert l.mxfp4_cache_copy(None, c, FAKE, FAKE, 1, None) == 1 == l.mxfp4_cache_copy(c, None, FAKE, FAKE, 1, None)
    assert l.mxfp4_attention_prefix(c, b, None, *ATTN.values()) == 1
    assert l.mxfp4_pages_compact_workspace_bytes(None) == -1 == l.mxfp4_pages_reserve_workspace_bytes(None, 1)


def test_binding_refuses():
    """Host tensors, wrong types and shapes, before the library is called."""
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 2, dtype=torch.int32)
    y = torch.zeros(1, 2, 16, 32, dtype=torch.uint8)
    cache = nv.Mxfp4Cache(y, y, y, y)
    pages = nv.Mxfp4Pages(t, i, i, 16)
    for call in (lambda: nv.mxfp4_norm_rope(x), lambda: nv.mxfp4_norm_rope_append(cache, x, x, x, t, i, i),
                 lambda: nv.mxfp4_attention_prefix(x, cache, t, i, i, t, i, i), lambda: nv.mxfp4_pages_free(pages, i),
                 lambda: nv.mxfp4_pages_fork(pages, i, i), lambda: nv.mxfp4_pages_reserve(pages, i, i),
                 lambda: nv.mxfp4_pages_compact(pages), lambda: nv.mxfp4_cache_copy(cache, i, i),
                 lambda: nv.mxfp4_pages_free(None, i), lambda: nv.mxfp4_pages_compact_workspace_bytes(pages)):
        with pytest.raises(ValueError):
            call()


def test_sizes_of_the_records():
    """The binding's structs are laid out as the header's."""
    assert [ctypes.sizeof(s) for s in (mxfp4._CPrefix, mxfp4._CNorm, mxfp4._CRotation, mxfp4._CPages)] == [48, 16, 64, 64]
