"""GPU: norms whose eps leaves fp32's range, and heads that do not depend on those beside them."""
import numpy as np
import pytest

from tests import mx_ref, mx_seq_ref as ref, parity
from tests.test_gpu_mx_attention import Case
from tests.test_gpu_mx_rope import check, rotation

pytestmark = pytest.mark.gpu

EPS = [1e-300, 2.0 ** -126, 2.0 ** 99, 2.0 ** 101, 3.4e38, 3.5e38, 1e39, 1e45, 1e60, 1e300]


@pytest.mark.parametrize("eps", EPS)
def test_every_eps(gpu, eps):
    """Positive and finite is all that is asked of it: numbers around the ends of fp32's range and beyond
    them, with heads of every size and weights that bring the result back into bf16's range."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(7)
    x = rng.standard_normal((3, 7, 128))
    for h, scale in enumerate([1.0, 1e-30, 1e-11, 1e14, 1e19, 1e30, 2.0 ** 125]):
        x[:, h] *= scale
    bits = mx_ref.f64_to_bits(x)
    rot, freqs, which = rotation(gpu, 64)
    pos = np.array([[0], [9], [70000]], np.int32)
    xd, pd = parity.to_device_bf16(bits, gpu), torch.from_numpy(pos).to(gpu)
    w = mx_ref.f64_to_bits(1 + 0.2 * rng.standard_normal(128))
    for weight in (None, w):
        wd = None if weight is None else parity.to_device_bf16(weight, gpu)
        got = nv.mxfp4_norm_rope(xd, rot, pd, weight=wd, eps=eps)
        check(got, bits, ref.turns(pos, freqs, which), eps=eps, weight=weight)
        for h in range(7):  # without the others in its wave
            got = nv.mxfp4_norm_rope(xd[:, h:h + 1], rot, pd, weight=wd, eps=eps)
            check(got, bits[:, h:h + 1], ref.turns(pos, freqs, which), eps=eps, weight=weight)


@pytest.mark.parametrize("eps", [1e39, 1e60])
def test_queries_and_keys_of_an_append(gpu, eps):
    """Both by the same eps."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(9, 12)], dim=64, page=16, kv_heads=1)
    bits = mx_ref.f64_to_bits(np.random.default_rng(8).standard_normal((9, 1, 64)))
    d = parity.to_device_bf16(bits, gpu)
    q = nv.mxfp4_norm_rope_append(c.cache, d, d, d, c.table, c.seq, c.cu, eps=eps)
    check(q, bits, None, eps=eps)
    k = nv.mxfp4_cache_read(c.cache, c.table, c.seq, c.cu, 9)[0].double().cpu().numpy()
    want = ref.norm_rope(mx_ref.bits_to_f64(bits), eps=eps)[0]
    np.testing.assert_array_equal(k, mx_ref.round_trip(mx_ref.f64_to_bits(want)))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_head_does_not_depend_on_those_beside_it(gpu, dim):
    """Bit for bit: heads split differently over ranks come out the same, whatever else is in the row
    (zeros, numbers whose squares leave fp32, infinities, NaN)."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    g = torch.Generator(device="cuda").manual_seed(dim)
    tokens, heads = 400, 2 * 1024 // dim + 3
    x = torch.randn(tokens, heads, dim, generator=g, device=gpu).bfloat16()
    w = (1 + 0.2 * torch.randn(dim, generator=g, device=gpu)).bfloat16()
    rot = nv.mxfp4_rotation(dim, gpu)
    pos = torch.arange(tokens, dtype=torch.int32, device=gpu)
    want = nv.mxfp4_norm_rope(x, rot, pos, weight=w, eps=1e-6)
    for other in (0.0, 2.0 ** 120, 2.0 ** -100, float("inf"), float("nan")):
        y = x.clone()
        y[:, 1::2] = other
        got = nv.mxfp4_norm_rope(y, rot, pos, weight=w, eps=1e-6)
        assert torch.equal(got[:, ::2], want[:, ::2]), other
    for h in (0, 1, heads - 1):
        alone = nv.mxfp4_norm_rope(x[:, h:h + 1], rot, pos, weight=w, eps=1e-6)
        assert torch.equal(alone, want[:, h:h + 1]), h
