"""GPU: attention over the MXFP4 cache where scale * score is large: every finite scale is allowed,
and what counts is the difference of the scores, not their size."""
import numpy as np
import pytest

from tests import mx_ref, parity
from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


def exact_scores(gpu, c, seed):
    """Keys and queries whose products and sums fp32 holds exactly: keys of E2M1 values with 4 at
    element 0, queries with eight whole numbers and 0, 2^20 or -2^20 at element 0, by row and head.
    So the scores are multiples of 1/2 up to 2^22 + 100, which need 24 bits."""
    rng = np.random.default_rng(seed)
    k = rng.choice(mx_ref.MAGNITUDES, c.k_bits.shape) * rng.choice([-1.0, 1.0], c.k_bits.shape)
    k[..., 0] = 4.0
    q = np.zeros(c.q_bits.shape)
    for row in q.reshape(-1, c.dim):
        row[1 + rng.permutation(c.dim - 1)[:8]] = rng.integers(-2, 3, 8)
    q[..., 0] = np.array([0.0, 2.0 ** 20, -2.0 ** 20])[np.arange(q[..., 0].size).reshape(q.shape[:2]) % 3]
    c.k_bits, c.q_bits = mx_ref.f64_to_bits(k), mx_ref.f64_to_bits(q)
    assert (mx_ref.round_trip(c.k_bits) == k).all() and (mx_ref.bits_to_f64(c.q_bits) == q).all()
    c.q = parity.to_device_bf16(c.q_bits, gpu)
    return c.fill(gpu)


def check(c, out, scale):
    """The scores are exact, so only what follows them counts: the exponent of a weight that is not
    below 2^-150 is within 3 roundings of 2^-24 and that of log2 e, each of at most 150, which is
    2^-14.5 of the weight in all; a weight and the sum are rounded to bf16 as everywhere (2^-8
    of sum w |v| + |o|); sums of at most 1000 tokens in fp32 (2^-24 each) and exp2: 2^-13.9; one
    rounding of the output. Weights below 2^-126 may be 0."""
    import torch
    k, v = (torch.from_numpy(mx_ref.round_trip(b)) for b in (c.k_bits, c.v_bits))
    q = torch.from_numpy(mx_ref.bits_to_f64(c.q_bits))
    got = out.double().cpu()
    at = base = 0
    for n, kv in c.lens:
        assert kv <= 1000
        args = (q[at:at + n], k[base:base + kv])
        vv = v[base:base + kv]
        o = mx_ref.attention(*args, vv, scale)[0]
        size = mx_ref.attention(*args, vv.abs(), scale)[0]
        tol = (2.0 ** -8 + 2.0 ** -13) * (size + o.abs()) + 2.0 ** -8 * o.abs() + 2.0 ** -110
        off = (got[at:at + n] - o).abs()
        assert bool((off <= tol).all()), (n, kv, int((~(off <= tol)).sum()), off.numel())
        at, base = at + n, base + kv


# 0.1733: scale * 2^22 * log2 e is 2^20 to four digits
@pytest.mark.parametrize("scale", [0.1733, 0.5, 4096.0, 1e8, 1e9, 1e20, 1e38])
@pytest.mark.parametrize("kw,lens", [(dict(group=6), [(1, 700), (2, 90), (1, 1)]), (dict(group=10, dim=64), [(3, 500)]),
                                     (dict(group=3, dim=256), [(1, 300), (4, 64)]), (dict(group=2), [(80, 300), (33, 33)]),
                                     (dict(group=2, dim=64, kv_heads=1), [(100, 700), (1, 90)]),
                                     (dict(group=2, dim=256, kv_heads=1), [(70, 130)])])
def test_large_scores(gpu, kw, lens, scale):
    """Both forms, whole, in pieces, and (16,384 with several sequences) both in one call."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = exact_scores(gpu, Case(gpu, lens, **kw), len(lens))
    for max_kv in (1, 1000, 1 << 14):
        check(c, nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, scale=scale, max_kv=max_kv), scale)


@pytest.mark.parametrize("q,kv", [(1, 700), (80, 300)])
@pytest.mark.parametrize("scale", [0.5, 1e6, 1e30])
def test_large_scores_that_rise(gpu, q, kv, scale):
    """Element 0 of the keys grows along the cache, so that one row's maximum goes from small
    scores to large ones, or comes down from them."""
    import nvfp4_block_scaled_swiglu_amd as nv
    for sign in (1, -1):
        c = Case(gpu, [(q, kv)], group=3, kv_heads=1)
        step = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0])[np.arange(kv) * 7 // kv][::sign]
        exact_scores(gpu, c, 5)
        k = mx_ref.bits_to_f64(c.k_bits)
        k[..., 0] = step[:, None]
        k[..., 1] = 4.0  # the block's scale stays 1
        c.k_bits = mx_ref.f64_to_bits(k)
        assert (mx_ref.round_trip(c.k_bits) == k).all()
        c.fill(gpu)
        for max_kv in (1, 1 << 14):
            check(c, nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, scale=scale, max_kv=max_kv), scale)


@pytest.mark.parametrize("exponent", [80, -100])
@pytest.mark.parametrize("lens", [[(1, 900), (3, 40)], [(60, 700)]])
def test_values_far_from_one(gpu, lens, exponent):
    """Values whose weighted sums are near the ends of what fp32 holds."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, group=3)
    c.v_bits = mx_ref.f64_to_bits(np.clip(mx_ref.bits_to_f64(c.v_bits) / 8, -1, 1) * 2.0 ** exponent)
    c.fill(gpu)
    for max_kv in (1, 1 << 14):
        c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=max_kv))
