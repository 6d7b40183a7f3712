"""Host-side checks of the MXFP4 operators (no GPU): the library exports what include/mxfp4.h
declares, sizes agree with the layout, every refusal returns its status before a device is
touched, and the tests' own statement of the format agrees with brute force."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest

import nvfp4_block_scaled_swiglu_amd as nv
from nvfp4_block_scaled_swiglu_amd import mxfp4
from tests import mx_ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mxfp4.h")
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


def test_binding_declares_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mxfp4_[a-z0-9_]+)\s*\(", text))
    assert names == set(mxfp4.SIGNATURES) and "mxfp4_attention" in names
    for n in names:
        assert hasattr(nv.lib(), n), n


@pytest.mark.parametrize("rows,k", [(0, 32), (1, 32), (1, 5376), (128, 128), (129, 160), (37810, 14336)])
def test_sizes(rows, k):
    cols = -(-(k // 32) // 4) * 4
    assert nv.mxfp4_qdata_bytes(rows, k) == rows * k // 2
    assert nv.mxfp4_scale_cols(k) == cols
    assert nv.mxfp4_scale_bytes(rows, k) == -(-rows // 128) * 128 * cols
    assert nv.mxfp4_scale_bytes(-1, k) == -1 and nv.mxfp4_qdata_bytes(rows, -1) == -1


def test_layout_statement():
    rows, cols = 200, 7
    s = np.arange(rows * cols, dtype=np.int64).reshape(rows, cols) % 251 + 1
    t = mx_ref.tiled(s.astype(np.uint8))
    assert t.size == 256 * 8
    for r, c in [(0, 0), (0, 6), (31, 3), (32, 0), (127, 5), (128, 1), (199, 6)]:
        at = ((r >> 7) * 2 + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3)
        assert t[at] == s[r, c]
    assert int((t != 0).sum()) == rows * cols


def test_format_statement_against_fractions():
    """The test oracle's codes against exact rationals, subnormals, ties and saturation included."""
    rng = np.random.default_rng(0)
    blocks = [rng.integers(0, 65536, 32), rng.integers(0, 0x100, 32), np.full(32, 0x8000)]
    blocks.append(np.array([0x40E0, 0x40C0, 0x40A0, 0x4060, 0x4020, 0x3FE0, 0x3FA0, 0x3F40] * 4))  # ties at scale 1
    blocks.append(rng.integers(0x3F00, 0x4300, 32) | (rng.integers(0, 2, 32) << 15))
    for b in blocks:
        b = np.where((b & 0x7F80) == 0x7F80, b & 0x807F, b).astype(np.uint16)
        codes, scale = mx_ref.quantize(b)
        x = [Fraction(float(v)) for v in mx_ref.bits_to_f64(b)]
        top = max(abs(v) for v in x)
        e = -127
        if top:
            f = 0
            while Fraction(2) ** (f + 1) <= top:
                f += 1
            while Fraction(2) ** f > top:
                f -= 1
            e = max(f - 2, -127)
        assert scale[0] == e + 127
        for i, v in enumerate(x):
            y = min(abs(v) / Fraction(2) ** e, Fraction(6))
            d = [abs(y - Fraction(float(m))) for m in mx_ref.MAGNITUDES]
            near = [c for c in range(8) if d[c] == min(d)]
            want = near[0] if len(near) == 1 else [c for c in near if c % 2 == 0][0]
            got = (codes[i // 2] >> (4 * (i % 2))) & 15
            assert got == want + 8 * (int(b[i]) >> 15)


def call(name, order, defaults, kw):
    args = dict(defaults)
    args.update(kw)
    return getattr(nv.lib(), name)(*[args[n] for n in order])


QUANT = dict(x=FAKE, ld=64, rows=16, k=64, q=FAKE, s=FAKE, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(rows=-1), 1), (dict(k=0), 1), (dict(k=48), 2),
    (dict(k=-32), 1), (dict(ld=32), 1), (dict(ld=68), 3), (dict(x=FAKE + 2), 3), (dict(q=FAKE + 4), 3), (dict(s=FAKE + 8), 3),
    (dict(k=1 << 24, ld=1 << 24), 2), (dict(ld=1 << 24), 2), (dict(rows=1 << 41), 2),
])
def test_quantize_refusals(kw, status):
    assert call("mxfp4_quantize", QUANT, QUANT, kw) == status
    assert nv.lib().nvfp4_last_error().decode() != ""


SWIGLU = dict(g=FAKE, ldg=64, u=FAKE, ldu=64, m=16, k=64, q=FAKE, s=FAKE, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(u=None), 1), (dict(ldu=16), 1), (dict(ldg=68), 3), (dict(u=FAKE + 2), 3), (dict(k=40), 2),
    (dict(s=None), 1),
])
def test_swiglu_refusals(kw, status):
    assert call("mxfp4_quantize_swiglu", SWIGLU, SWIGLU, kw) == status


DEQUANT = dict(q=FAKE, s=FAKE, rows=16, k=64, y=FAKE, ld=64, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(y=None), 1), (dict(k=16), 2), (dict(ld=56), 1), (dict(ld=66), 3), (dict(y=FAKE + 8), 3),
])
def test_dequantize_refusals(kw, status):
    assert call("mxfp4_dequantize", DEQUANT, DEQUANT, kw) == status


GEMM = dict(aq=FAKE, as_=FAKE, wq=FAKE, ws=FAKE, d=FAKE, ld=16, m=16, n=16, k=64, st=None)


@pytest.mark.parametrize("kw,status", [
    (dict(aq=None), 1), (dict(as_=None), 1), (dict(wq=None), 1), (dict(ws=None), 1), (dict(d=None), 1), (dict(m=-1), 1),
    (dict(n=0), 1), (dict(k=0), 1), (dict(k=80), 2), (dict(ld=15), 1), (dict(d=FAKE + 1), 3), (dict(ws=FAKE + 4), 3),
    (dict(m=1 << 35), 2), (dict(m=1 << 19, n=1 << 19, ld=1 << 19), 2),
])
def test_gemm_refusals(kw, status):
    assert call("mxfp4_gemm_bf16out", GEMM, GEMM, kw) == status


CACHE = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=4, size=16, heads=2, dim=64)
BATCH = dict(table=FAKE, lens=FAKE, cu=FAKE, batch=2, pages=2, stride=2, tokens=8)


def structs(kw):
    c, b = dict(CACHE), dict(BATCH)
    c.update({n[2:]: v for n, v in kw.items() if n.startswith("c_")})
    b.update({n[2:]: v for n, v in kw.items() if n.startswith("b_")})
    return mxfp4._CCache(*c.values()), mxfp4._CBatch(*b.values())


CACHE_REFUSALS = [
    (dict(c_kc=None), 1), (dict(c_vs=None), 1), (dict(c_ks=FAKE + 8), 3), (dict(c_pages=0), 1), (dict(c_size=24), 2),
    (dict(c_size=8), 2), (dict(c_size=65536), 2), (dict(c_heads=0), 1), (dict(c_heads=2000), 2), (dict(c_dim=96), 2),
    (dict(c_dim=-64), 1), (dict(b_table=None), 1), (dict(b_lens=None), 1), (dict(b_cu=None), 1), (dict(b_cu=FAKE + 2), 3),
    (dict(b_batch=-1), 1), (dict(b_tokens=-1), 1), (dict(b_stride=1), 1), (dict(b_tokens=1 << 31), 2),
    (dict(b_pages=1 << 26, b_stride=1 << 26, c_size=16), 2),
]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 2), 3), (dict(kt=-8), 1), (dict(vh=60), 3), (dict(kt=1 << 32), 2),
])
def test_cache_refusals(kw, status):
    c, b = structs(kw)
    order = dict(k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64)
    args = {**order, **{n: v for n, v in kw.items() if n in order}}
    for name in ("mxfp4_cache_append", "mxfp4_cache_read"):
        assert getattr(nv.lib(), name)(c, b, *args.values(), None) == status, name


def test_cache_read_refuses_rows_in_one_another():
    c, b = structs({})
    f = nv.lib().mxfp4_cache_read
    assert f(c, b, FAKE, 64, 64, FAKE, 128, 64, None) == 1
    assert f(c, b, FAKE, 128, 64, FAKE, 0, 64, None) == 1
    assert f(None, b, FAKE, 128, 64, FAKE, 128, 64, None) == 1
    assert nv.lib().mxfp4_cache_append(c, None, FAKE, 128, 64, FAKE, 128, 64, None) == 1


ATTN = dict(q=FAKE, qt=256, qh=64, heads=4, scale=0.125, causal=1, window=0, sinks=0, kv=32, out=FAKE, ot=256, oh=64,
            ws=None, wb=0, st=None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS + [
    (dict(q=None), 1), (dict(out=None), 1), (dict(heads=3), 1), (dict(heads=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1), (dict(window=-1), 1),
    (dict(sinks=4), 1), (dict(causal=0, window=8), 1), (dict(window=8, sinks=-1), 1), (dict(kv=0), 1), (dict(qh=60), 3),
    (dict(out=FAKE + 8), 3), (dict(ot=64), 1), (dict(oh=0), 1), (dict(heads=1 << 17), 2), (dict(kv=1 << 20), 4),
    (dict(kv=1 << 20, ws=FAKE, wb=64), 4), (dict(kv=1 << 20, ws=FAKE + 4, wb=1 << 30), 3),
])
def test_attention_refusals(kw, status):
    c, b = structs(kw)
    args = {**ATTN, **{n: v for n, v in kw.items() if n in ATTN}}
    assert nv.lib().mxfp4_attention(c, b, *args.values()) == status
    assert nv.lib().nvfp4_last_error().decode() != ""


def test_attention_workspace():
    """No workspace for short caches; with splits, room for a float row and two floats each."""
    f = nv.lib().mxfp4_attention_workspace_bytes
    c, b = structs({})
    assert f(c, b, 4, 32, 0, 0) == 0
    size = f(c, b, 4, 1 << 17, 0, 0)
    assert size > 0 and size % (8 * 4 * (64 + 2) * 4) == 0
    assert f(c, b, 4, 1 << 17, 64, 4) == 0  # a short window: nothing to split
    assert f(c, b, 3, 32, 0, 0) == -1 and f(c, b, 4, 0, 0, 0) == -1
    c, b = structs(dict(b_tokens=0))
    assert f(c, b, 4, 1 << 17, 0, 0) == 0


def test_valid_calls_without_gpu_report_no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    c, b = structs({})
    l = nv.lib()
    assert call("mxfp4_quantize", QUANT, QUANT, {}) == 5
    assert call("mxfp4_quantize_swiglu", SWIGLU, SWIGLU, {}) == 5
    assert call("mxfp4_dequantize", DEQUANT, DEQUANT, {}) == 5
    assert call("mxfp4_gemm_bf16out", GEMM, GEMM, {}) == 5
    assert l.mxfp4_cache_append(c, b, FAKE, 128, 64, FAKE, 128, 64, None) == 5
    assert l.mxfp4_cache_read(c, b, FAKE, 128, 64, FAKE, 128, 64, None) == 5
    assert l.mxfp4_attention(c, b, *ATTN.values()) == 5


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(x)
    with pytest.raises(ValueError):
        nv.mxfp4_quantize_swiglu(x, x)
    with pytest.raises(ValueError):
        nv.mxfp4_dequantize(x)
    t = nv.Mxfp4Tensor(x, x, 4, 64)
    with pytest.raises(ValueError):
        nv.mxfp4_gemm_bf16out(t, t)
    cache = nv.Mxfp4Cache(x, x, x, x)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.mxfp4_attention(x, cache, i, i, i)
    with pytest.raises(ValueError):
        nv.mxfp4_cache_append(cache, x, x, i, i, i)
