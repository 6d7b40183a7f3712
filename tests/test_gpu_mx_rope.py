"""GPU: norms and rotation of heads, and the append behind them, against float64 with exact angles."""
import numpy as np
import pytest

from tests import mx_ref, mx_seq_ref as ref, parity
from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


def rotation(gpu, rotary, axes=1, interleaved=False, seed=0):
    """(the library's rotation, freqs, axes of the pairs)"""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(seed)
    freqs = (10000.0 ** -rng.random(rotary // 2)).astype(np.float32)
    which = rng.integers(0, axes, rotary // 2).astype(np.int32)
    return nv.Mxfp4Rotation(torch.from_numpy(freqs).to(gpu), torch.from_numpy(which).to(gpu), axes, interleaved), freqs, which


def check(got, bits, angle, interleaved=False, eps=None, weight=None):
    y, size = ref.norm_rope(mx_ref.bits_to_f64(bits), angle, interleaved, eps, None if weight is None else mx_ref.bits_to_f64(weight))
    got = got.double().cpu().numpy()
    nan = np.isnan(y)
    np.testing.assert_array_equal(np.isnan(got), nan)
    off = np.where(nan, 0.0, np.abs(got - y))
    tol = np.where(nan, 1.0, ref.norm_rope_tolerance(y, size))
    assert (off <= tol).all(), (float((off / tol).max()), int((off > tol).sum()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary,heads,tokens,axes", [
    (64, 64, 1, 1, 1), (64, 16, 17, 3, 2), (64, 48, 5, 4, 3), (128, 128, 8, 5, 1), (128, 32, 3, 7, 3), (128, 96, 9, 2, 4),
    (256, 256, 4, 3, 2), (256, 64, 5, 5, 1), (256, 240, 1, 2, 5), (128, 128, 70, 33, 3),
])
def test_norm_and_rotation(gpu, dim, rotary, heads, tokens, axes, interleaved):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(dim + rotary + heads)
    rot, freqs, which = rotation(gpu, rotary, axes, interleaved)
    pos = rng.integers(-5, 300000, (tokens, axes)).astype(np.int32)
    bits = mx_ref.f64_to_bits(rng.standard_normal((tokens, heads, dim)) * 3)
    w = mx_ref.f64_to_bits(1 + 0.2 * rng.standard_normal(dim))
    x, wd, pd = parity.to_device_bf16(bits, gpu), parity.to_device_bf16(w, gpu), torch.from_numpy(pos).to(gpu)
    angle = ref.turns(pos, freqs, which)
    check(nv.mxfp4_norm_rope(x, rot, pd, weight=wd, eps=1e-6), bits, angle, interleaved, 1e-6, w)
    check(nv.mxfp4_norm_rope(x, rot, pd, eps=1e-3), bits, angle, interleaved, 1e-3)
    check(nv.mxfp4_norm_rope(x, rot, pd), bits, angle, interleaved)
    check(nv.mxfp4_norm_rope(x, weight=wd, eps=1e-6), bits, None, eps=1e-6, weight=w)
    assert torch.equal(nv.mxfp4_norm_rope(x), x)
    # one position for every axis; positions by axis first
    check(nv.mxfp4_norm_rope(x, rot, pd[:, 0].contiguous()), bits, ref.turns(pos[:, :1], freqs), interleaved)
    check(nv.mxfp4_norm_rope(x, rot, pd.t().contiguous().t()), bits, angle, interleaved)
    # heads in a wider row, heads first, and in place
    wide = torch.full((tokens, 3 * heads, dim), 7.0, dtype=torch.bfloat16, device=gpu)
    wide[:, heads:2 * heads] = x
    want = nv.mxfp4_norm_rope(x, rot, pd, weight=wd, eps=1e-6)
    first = torch.empty((heads, tokens, dim), dtype=torch.bfloat16, device=gpu).transpose(0, 1)
    assert nv.mxfp4_norm_rope(wide[:, heads:2 * heads], rot, pd, weight=wd, eps=1e-6, out=first) is first
    assert torch.equal(first, want)
    nv.mxfp4_norm_rope(wide[:, heads:2 * heads], rot, pd, weight=wd, eps=1e-6, out=wide[:, heads:2 * heads])
    assert torch.equal(wide[:, heads:2 * heads], want)
    assert bool((wide[:, :heads] == 7).all()) and bool((wide[:, 2 * heads:] == 7).all())


def test_values_at_the_edges_of_the_types(gpu):
    """Heads of zeros, of numbers whose squares leave fp32, with an infinity, with a NaN: each alone."""
    import nvfp4_block_scaled_swiglu_amd as nv
    import torch
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 9, 128))
    for h, scale in enumerate([0.0, 1e-38, 1e-30, 1e-20, 1.0, 1e19, 1e30, 2.0 ** 125, 1.0]):
        x[:, h] *= scale
    bits = mx_ref.f64_to_bits(x)
    bits[0, 4, 17], bits[0, 8, 3], bits[1, 8, 100] = 0x7F80, 0x7FC0, 0xFF80
    rot, freqs, which = rotation(gpu, 64)
    pos = np.array([[5], [123456]], np.int32)
    xd, pd = parity.to_device_bf16(bits, gpu), torch.from_numpy(pos).to(gpu)
    for eps in (1e-6, 1e-30, 1e30, 5e-324):
        # (an infinite head: its norm is infinite, others 0, itself NaN, and its pair with it)
        check(nv.mxfp4_norm_rope(xd, rot, pd, eps=eps), bits, ref.turns(pos, freqs, which), eps=eps)


@pytest.mark.parametrize("position", [0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(gpu, position):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(1)
    freqs = np.concatenate([[1.0, 0.5, 3.0, 1e-5, 0.0, 0.99999994, 2.0 ** -20, 1e3], rng.random(24)]).astype(np.float32)
    rot = nv.Mxfp4Rotation(torch.from_numpy(freqs).to(gpu))
    pos = np.array([[position]], np.int64)
    bits = mx_ref.f64_to_bits(rng.standard_normal((1, 4, 64)))
    got = nv.mxfp4_norm_rope(parity.to_device_bf16(bits, gpu), rot, torch.tensor([position], dtype=torch.int32, device=gpu))
    check(got, bits, ref.turns(pos, freqs))


def test_axes_out_of_range_are_clamped(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rot, freqs, _ = rotation(gpu, 64, 2)
    which = np.array([-7, 0, 1, 2, 2 ** 31 - 1, -2 ** 31, 1, 0] * 4, np.int32)
    rot = nv.Mxfp4Rotation(rot.freqs, torch.from_numpy(which).to(gpu), 2)
    pos = np.array([[3, 1000], [77, 5]], np.int32)
    bits = mx_ref.f64_to_bits(np.random.default_rng(0).standard_normal((2, 2, 64)))
    got = nv.mxfp4_norm_rope(parity.to_device_bf16(bits, gpu), rot, torch.from_numpy(pos).to(gpu))
    check(got, bits, ref.turns(pos, freqs, np.clip(which, 0, 1)))


def test_many_rows(gpu):
    """A wave to a token (more than 2,048 of them), heads that do not fill its steps; rows drawn."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    g = torch.Generator(device="cuda").manual_seed(0)
    tokens, heads, dim = 5003, 13, 128
    x = torch.randn(tokens, heads, dim, generator=g, device=gpu).bfloat16()
    rot, freqs, which = rotation(gpu, 128, 3, True)
    pos = torch.randint(0, 5000, (tokens, 3), generator=g, device=gpu, dtype=torch.int32)
    got = nv.mxfp4_norm_rope(x, rot, pos, eps=1e-6)
    at = np.random.default_rng(0).permutation(tokens)[:40]
    at[0], at[1] = 0, tokens - 1
    check(got[at], parity.tensor_bits(x[at].contiguous()), ref.turns(pos[at].cpu().numpy(), freqs, which), True, 1e-6)


def usual(gpu):
    import nvfp4_block_scaled_swiglu_amd as nv
    return nv.mxfp4_rotation(128, gpu, theta=1e6, sections=[16, 24, 24])


def test_usual_rotations(gpu):
    import nvfp4_block_scaled_swiglu_amd as nv
    r = usual(gpu)
    assert r.axis_count == 3 and r.axes.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    np.testing.assert_allclose(r.freqs.cpu().numpy(), 1e6 ** -(np.arange(64) / 64), rtol=2.0 ** -23)
    r = nv.mxfp4_rotation(128, gpu, sections=[22, 21, 21], separate=True, interleaved=True)
    want = np.concatenate([1e4 ** -(np.arange(n) / n) for n in (22, 21, 21)])
    np.testing.assert_allclose(r.freqs.cpu().numpy(), want, rtol=2.0 ** -23)
    assert r.interleaved and nv.mxfp4_rotation(64, gpu).axes is None
    for bad in (dict(sections=[16, 24]), dict(sections=[]), dict(sections=[-1, 65])):
        with pytest.raises(ValueError):
            nv.mxfp4_rotation(128, gpu, **bad)


APPENDS = [
    (dict(dim=128, page=16), 128, [(1, 1), (3, 17), (0, 5), (20, 20)]),
    (dict(dim=128, page=64, kv_heads=8), 32, [(1, n) for n in range(1, 70)]),
    (dict(dim=64, page=32, kv_heads=3), 48, [(33, 64), (2, 31), (65, 65)]),
    (dict(dim=256, page=128, kv_heads=1), 64, [(1, 300), (130, 131)]),
    (dict(dim=256, page=16, kv_heads=5), 256, [(7, 30)]),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kw,rotary,lens", APPENDS)
def test_append(gpu, kw, rotary, lens, interleaved):
    """q by its tolerance; the cache byte for byte, what is not written among it."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, group=3, **kw)
    rng = np.random.default_rng(11)
    rot, freqs, which = rotation(gpu, rotary, 3, interleaved)
    pos = rng.integers(0, 200000, (c.tokens, 3)).astype(np.int32)
    own = np.concatenate([np.arange(kv - q, kv) for q, kv in lens])[:, None]
    width = c.heads + 2 * c.kv_heads
    qkv = mx_ref.f64_to_bits(rng.standard_normal((c.tokens, width, c.dim)) * 2)
    ws = [mx_ref.f64_to_bits(1 + 0.2 * rng.standard_normal(c.dim)) for _ in range(2)]
    wd = [parity.to_device_bf16(w, gpu) for w in ws]
    parts = [slice(0, c.heads), slice(c.heads, c.heads + c.kv_heads), slice(c.heads + c.kv_heads, width)]
    packed = parity.to_device_bf16(qkv, gpu)
    for given, eps, weights in ((True, 1e-6, True), (False, 1e-5, False), (False, None, False)):
        want = [t.cpu().numpy().copy() for t in (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)]
        got = nv.mxfp4_norm_rope_append(c.cache, *(packed[:, p] for p in parts), c.table, c.seq, c.cu, rot,
                                        torch.from_numpy(pos).to(gpu) if given else None,
                                        q_weight=wd[0] if weights else None, k_weight=wd[1] if weights else None, eps=eps)
        angle = ref.turns(pos if given else own, freqs, which if given else None)
        check(got, qkv[:, parts[0]], angle, interleaved, eps, ws[0] if weights else None)
        k, _ = ref.norm_rope(mx_ref.bits_to_f64(qkv[:, parts[1]]), angle, interleaved, eps,
                             mx_ref.bits_to_f64(ws[1]) if weights else None)
        k = mx_ref.f64_to_bits(k)
        row = 0
        for i, (n, kv) in enumerate(lens):
            for t in range(kv - n, kv):
                p, s = c.table_np[i, t // c.page], t % c.page
                for j, b in ((0, k[row]), (2, qkv[row, parts[2]])):
                    want[j][p, :, s], want[j + 1][p, :, s] = mx_ref.quantize(b)
                row += 1
        for t, w in zip((c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales), want):
            np.testing.assert_array_equal(t.cpu().numpy(), w)


def test_append_without_change_is_the_plain_append(gpu):
    """Neither norm nor rotation, and no queries: mxfp4_cache_append, NaN and infinities among the values."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    caches = []
    for whole in (False, True):
        c = Case(gpu, [(9, 40), (30, 30)], dim=128, page=16, kv_heads=3)
        rng = np.random.default_rng(2)
        bits = [mx_ref.f64_to_bits(rng.standard_normal((c.tokens, 3, 128))) for _ in range(2)]
        bits[0][4, 1, 9], bits[0][5, 0, 40], bits[1][6, 2, 0] = 0x7F80, 0x7FC1, 0xFFC0
        bits[0][7, :, :] = 0x8000
        k, v = (parity.to_device_bf16(b, gpu) for b in bits)
        if whole:
            nv.mxfp4_cache_append(c.cache, k, v, c.table, c.seq, c.cu)
        else:
            q = torch.empty((c.tokens, 0, 128), dtype=torch.bfloat16, device=gpu)
            assert nv.mxfp4_norm_rope_append(c.cache, q, k, v, c.table, c.seq, c.cu).shape == q.shape
        caches.append(c.cache)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)), n


def test_keys_at_the_edges_of_the_types(gpu):
    """Through the append: keys of zeros, of numbers at either end of the range, with an infinity or a NaN."""
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 1, 64))
    for i, scale in enumerate([0.0, 1e-38, 1e-30, 1e-20, 1.0, 1e19, 1e30, 2.0 ** 125, 1.0]):
        x[i] *= scale
    bits = mx_ref.f64_to_bits(x)
    bits[4, 0, 17], bits[8, 0, 3] = 0xFF80, 0x7FC0
    rot, freqs, _ = rotation(gpu, 64)
    rot.axes = None
    d = parity.to_device_bf16(bits, gpu)
    for eps in (1e-6, 1e-30, 1e30, 5e-324):
        c = Case(gpu, [(9, 12)], dim=64, page=16, kv_heads=1)
        nv.mxfp4_norm_rope_append(c.cache, d, d, d, c.table, c.seq, c.cu, rot, eps=eps)
        k = nv.mxfp4_cache_read(c.cache, c.table, c.seq, c.cu, 9)[0].double().cpu().numpy()
        y, _ = ref.norm_rope(mx_ref.bits_to_f64(bits), ref.turns(np.arange(3, 12)[:, None], freqs), eps=eps)
        broken = [4, 8]
        fine = [i for i in range(9) if i not in broken]
        np.testing.assert_array_equal(k[fine], mx_ref.round_trip(mx_ref.f64_to_bits(y[fine])))
        # the infinity: NaN for its block and its pair's; the NaN: for all of the head
        assert np.isnan(k[8]).all() and np.isnan(k[4]).all()


def test_rows_without_a_place(gpu):
    """Rows behind the last sequence and before the first, sequences shorter than their rows, pages that
    are not there: caches keep their bytes, rows of no sequence their q."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(4, 2), (6, 6), (3, 40)], dim=64, page=16, kv_heads=2)
    c.table[2, 2] = c.cache.num_pages  # of the last sequence's positions 37, 38, 39: page 2 is not there
    tokens = 3 + 13 + 5
    cu = c.cu + 3
    rng = np.random.default_rng(4)
    bits = [mx_ref.f64_to_bits(rng.standard_normal((tokens, 2, 64))) for _ in range(3)]
    q, k, v = (parity.to_device_bf16(b, gpu) for b in bits)
    rot, freqs, _ = rotation(gpu, 64)
    rot.axes = None
    before = [t.clone() for t in (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)]
    out = torch.full_like(q, 9.0)
    nv.mxfp4_norm_rope_append(c.cache, q, k, v, c.table, c.seq, cu, rot, eps=1e-6, out=out)
    assert bool((out[:3] == 9).all()) and bool((out[16:] == 9).all())
    pos = np.array([-2, -1, 0, 1, 0, 1, 2, 3, 4, 5, 37, 38, 39])[:, None]
    check(out[3:16], bits[0][3:16], ref.turns(pos, freqs), eps=1e-6)
    want = [t.cpu().numpy() for t in before]
    kk = mx_ref.f64_to_bits(ref.norm_rope(mx_ref.bits_to_f64(bits[1][3:16]), ref.turns(pos, freqs), eps=1e-6)[0])
    for row, (seq, t) in {2: (0, 0), 3: (0, 1), **{4 + i: (1, i) for i in range(6)}}.items():
        p, s = c.table_np[seq, t // 16], t % 16
        for j, b in ((0, kk[row]), (2, bits[2][3 + row])):
            want[j][p, :, s], want[j + 1][p, :, s] = mx_ref.quantize(b)
    for t, w in zip((c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales), want):
        np.testing.assert_array_equal(t.cpu().numpy(), w)


@pytest.mark.parametrize("batch", [1, 2, 63, 64, 65, 200, 4097])
def test_search_for_the_sequence(gpu, batch):
    """Batches around the powers of 64 that the search goes by, empty sequences among them."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(batch)
    n = rng.integers(0, 3, batch)
    n[rng.integers(batch)] = 2
    kv = n + rng.integers(0, 14, batch)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    tokens = int(cu[-1])
    cache = nv.empty_mxfp4_cache(batch, 16, 1, 64, gpu)
    table = rng.permutation(batch).astype(np.int32)[:, None]
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.zero_()
    x = np.arange(1, tokens + 1)[:, None, None] * np.ones((1, 1, 64))
    bits = mx_ref.f64_to_bits(x)
    d = parity.to_device_bf16(bits, gpu)
    nv.mxfp4_norm_rope_append(cache, d, d, d, *(torch.from_numpy(t.astype(np.int32)).to(gpu) for t in (table, kv, cu)))
    want = np.zeros((batch, 1, 16, 32), np.uint8), np.zeros((batch, 1, 16, 2), np.uint8)
    for b in range(batch):
        for i in range(n[b]):
            at = (table[b, 0], 0, kv[b] - n[b] + i)
            want[0][at], want[1][at] = mx_ref.quantize(bits[cu[b] + i, 0])
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        np.testing.assert_array_equal(codes.cpu().numpy(), want[0])
        np.testing.assert_array_equal(scales.cpu().numpy(), want[1])
