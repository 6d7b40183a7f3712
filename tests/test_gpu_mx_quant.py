"""GPU: MXFP4 quantization (plain, SwiGLU) and its reverse, byte for byte against the tests' own
statement of the format."""
import numpy as np
import pytest

import oracle
from tests import mx_ref, parity

pytestmark = pytest.mark.gpu


def bits(rows, k, seed, special=False):
    """Normal values over many binades; with `special`, whole blocks of subnormals, zeros, huge
    values, infinities and NaN among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-20, 20, (rows, k // 32)).repeat(32, 1))
    b = mx_ref.f64_to_bits(x)
    if special:
        blocks = b.reshape(-1, 32)
        for i, kind in zip(rng.permutation(len(blocks))[:8], range(8)):
            if kind == 0:
                blocks[i] = rng.integers(0, 0x80, 32)                # subnormals
            elif kind == 1:
                blocks[i] = 0x8000 * rng.integers(0, 2, 32)           # zeros of both signs
            elif kind == 2:
                blocks[i, 5] = 0x7F80                                 # an infinity
            elif kind == 3:
                blocks[i, 31] = 0xFFC0                                # a NaN
            elif kind == 4:
                blocks[i] = rng.integers(0x7E00, 0x7F80, 32)          # up to the largest finite
            elif kind == 5:
                blocks[i] = 0x0080 + rng.integers(0, 0x200, 32)       # scale byte 0 and next to it
            elif kind == 6:
                blocks[i] = 0x3F80 + 8 * np.arange(32)                # every half step and tie
            else:
                blocks[i, 0] = 0xFF80
    return b


def unpack(t):
    return t.qdata.cpu().numpy(), t.scales.cpu().numpy()


def check(t, codes, scale):
    q, s = unpack(t)
    np.testing.assert_array_equal(q, codes)
    np.testing.assert_array_equal(s, mx_ref.tiled(scale))


SHAPES = [(1, 32), (1, 5376), (3, 64), (17, 96), (127, 160), (128, 512), (129, 544), (300, 1120), (5, 14336)]


@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize_and_back(gpu, rows, k):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    b = bits(rows, k, rows + k, special=rows * k >= 32 * 64)
    x = parity.to_device_bf16(b, gpu)
    out = nv.empty_mxfp4(rows, k, gpu)
    out.qdata.fill_(0xA5)
    out.scales.fill_(0xA5)
    assert nv.mxfp4_quantize(x, out=out) is out
    codes, scale = mx_ref.quantize(b)
    check(out, codes, scale)
    y = nv.mxfp4_dequantize(out)
    want = mx_ref.values(codes, scale)
    got = y.double().cpu().numpy()
    np.testing.assert_array_equal(got, want)  # NaN in the same places; every value exact in bf16
    assert (np.signbit(got) == np.signbit(want))[~np.isnan(want)].all()
    # again on what came back: finite blocks whose largest value did not saturate downwards keep their bytes
    again = nv.mxfp4_quantize(torch.nan_to_num(y, 0.0, 0.0, 0.0))
    q2, s2 = mx_ref.quantize(parity.tensor_bits(torch.nan_to_num(y, 0.0, 0.0, 0.0)))
    check(again, q2, s2)


def test_every_bf16_value_at_every_place_of_a_block(gpu):
    """All 65,536 patterns, each alone in a block of zeros (its own scale) at a moving place."""
    import nvfp4_block_scaled_swiglu_amd as nv
    b = np.zeros((1024, 64, 32), np.uint16)
    v = np.arange(65536).reshape(1024, 64)
    np.put_along_axis(b, (v % 32)[:, :, None], v[:, :, None].astype(np.uint16), 2)
    b = b.reshape(1024, 2048)
    t = nv.mxfp4_quantize(parity.to_device_bf16(b, gpu))
    check(t, *mx_ref.quantize(b))


def test_strided_input_and_output(gpu):
    """Rows of a wider tensor in, rows of a wider tensor out; the rest stays as it was."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    b = bits(70, 512, 3)
    wide = parity.to_device_bf16(b, gpu)
    x = wide[2:67, 96:96 + 352]
    t = nv.mxfp4_quantize(x)
    codes, scale = mx_ref.quantize(b[2:67, 96:448])
    check(t, codes, scale)
    hold = torch.full((70, 512), 7.0, dtype=torch.bfloat16, device=gpu)
    y = nv.mxfp4_dequantize(t, out=hold[2:67, 96:448])
    np.testing.assert_array_equal(y.double().cpu().numpy(), mx_ref.values(codes, scale))
    rest = hold.clone()
    rest[2:67, 96:448] = 7.0
    assert (rest == 7.0).all()


def test_empty(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    t = nv.mxfp4_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device=gpu))
    assert t.rows == 0 and t.scales.numel() == 0 and nv.mxfp4_dequantize(t).shape == (0, 64)


def test_swiglu_every_gate(gpu):
    """y for all 65,280 finite gates under several ups: the oracle's correctly rounded silu, one
    product rounding, then the format."""
    import nvfp4_block_scaled_swiglu_amd as nv
    g = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    g = np.where((g & 0x7F80) == 0x7F80, 0x3F80, g).reshape(64, 1024)
    silu = oracle.silu_table()[g]
    for i, u in enumerate([0x3F80, 0xBF81, 0x0101, 0x7E7F, 0x3FFF]):
        up = np.full_like(g, u)
        y = mx_ref.f64_to_bits(mx_ref.bits_to_f64(silu) * mx_ref.bits_to_f64(up))
        t = nv.mxfp4_quantize_swiglu(parity.to_device_bf16(g, gpu), parity.to_device_bf16(up, gpu))
        check(t, *mx_ref.quantize(y))


@pytest.mark.parametrize("rows,k", [(1, 14336), (9, 96), (131, 1056)])
def test_swiglu(gpu, rows, k):
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(rows)
    gate = mx_ref.f64_to_bits(rng.standard_normal((rows, k)) * np.where(rng.random((1, k)) < 0.02, 20.0, 1.0))
    up = mx_ref.f64_to_bits(rng.standard_normal((rows, k)))
    silu = oracle.silu_table()[gate]
    y = mx_ref.f64_to_bits(mx_ref.bits_to_f64(silu) * mx_ref.bits_to_f64(up))
    t = nv.mxfp4_quantize_swiglu(parity.to_device_bf16(gate, gpu), parity.to_device_bf16(up, gpu))
    check(t, *mx_ref.quantize(y))


def test_swiglu_not_finite(gpu):
    """A gate or up that is not finite makes its block NaN and no other."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    gate, up = (torch.ones(4, 128, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    gate[0, 3] = float("nan")
    gate[1, 40] = float("inf")
    up[2, 100] = float("-inf")
    y = nv.mxfp4_dequantize(nv.mxfp4_quantize_swiglu(gate, up))
    want = torch.zeros(4, 128, dtype=torch.bool, device=gpu)
    want[0, :32] = want[1, 32:64] = want[2, 96:] = True
    assert torch.equal(torch.isnan(y), want)


def test_refusals(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=gpu)
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(x.float())
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        nv.mxfp4_quantize(x, out=nv.empty_mxfp4(5, 64, gpu))
    with pytest.raises(ValueError):
        nv.mxfp4_quantize_swiglu(x, x[:3])
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mxfp4_quantize(x[:, :48])
    assert e.value.status == 2
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mxfp4_quantize(x.reshape(-1)[4:4 + 32].reshape(1, 32))
    assert e.value.status == 3
    assert nv.mxfp4_quantize(x[:, :48], strict=False) is None
    assert nv.LAST_FALLBACK["mxfp4_quantize"][0] == 2
