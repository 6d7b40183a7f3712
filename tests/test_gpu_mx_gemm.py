"""GPU: the MXFP4 product against float64, over every kernel variant's sizes."""
import numpy as np
import pytest

from tests import mx_ref, parity

pytestmark = pytest.mark.gpu


def operand(rows, k, seed, gpu, sigma=1.0):
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * sigma * np.exp2(rng.integers(-3, 4, (rows, 1)))
    x[:, 7::100] *= 20
    b = mx_ref.f64_to_bits(x)
    return nv.mxfp4_quantize(parity.to_device_bf16(b, gpu)), mx_ref.round_trip(b)


def compare(got, a, w, k):
    ref, mags = mx_ref.product(a, w)
    off = np.abs(got.double().cpu().numpy() - ref)
    tol = mx_ref.product_tolerance(ref, mags, k)
    worst = np.unravel_index(np.argmax(off / tol), off.shape)
    assert (off <= tol).all(), (worst, off[worst], tol[worst], int((off > tol).sum()))


# few rows (one to four 16-row tiles), small tiles, large tiles; K of one block, odd numbers of
# blocks and whole steps; N that is odd, not a multiple of 8, of 16, of a tile
SHAPES = [(1, 16, 32), (1, 5376, 14336), (5, 77, 96), (16, 130, 128), (17, 64, 1056), (31, 33, 416), (48, 1000, 5376),
          (64, 250, 544), (65, 129, 160), (128, 128, 128), (200, 777, 2080), (1021, 300, 7168), (257, 1, 64),
          (4099, 4100, 288), (4096, 4352, 640), (4200, 4104, 32)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(gpu, m, n, k):
    import nvfp4_block_scaled_swiglu_amd as nv
    a, av = operand(m, k, m + n, gpu)
    w, wv = operand(n, k, m + n + 1, gpu, 0.02)
    out = nv.mxfp4_gemm_bf16out(a, w)
    compare(out, av, wv, k)
    assert (out == nv.mxfp4_gemm_bf16out(a, w)).all()  # the same order of sums every time


@pytest.mark.parametrize("m,n,k", [(7, 48, 256), (130, 264, 192), (4100, 4136, 160)])
def test_strided_output(gpu, m, n, k):
    """Rows of a wider tensor, 16-byte aligned and not; what lies around stays as it was."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    a, av = operand(m, k, 1, gpu)
    w, wv = operand(n, k, 2, gpu)
    for left, right in ((8, 24), (3, 2)):
        hold = torch.full((m + 2, left + n + right), 7.0, dtype=torch.bfloat16, device=gpu)
        out = hold[1:-1, left:left + n]
        assert nv.mxfp4_gemm_bf16out(a, w, out=out) is out
        compare(out, av, wv, k)
        rest = hold.clone()
        rest[1:-1, left:left + n] = 7.0
        assert (rest == 7.0).all()


@pytest.mark.parametrize("m", [1, 40, 200, 4200])
def test_exact_gather(gpu, m):
    """A weight of ones on a diagonal gives the activation's values, each exact in bf16; NaN blocks
    reach their own rows and the columns of their block... and no other row."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    k = 256
    rng = np.random.default_rng(m)
    x = mx_ref.f64_to_bits(rng.standard_normal((m, k)) * np.exp2(rng.integers(-60, 60, (m, 1))))
    x[0, 5] = 0x7F80 if m > 1 else x[0, 5]
    a = nv.mxfp4_quantize(parity.to_device_bf16(x, gpu))
    w = nv.mxfp4_quantize(torch.eye(k, dtype=torch.bfloat16, device=gpu).repeat(17, 1))
    got = nv.mxfp4_gemm_bf16out(a, w).double().cpu().numpy()
    want = np.tile(mx_ref.round_trip(x), (1, 17))
    if m > 1:
        assert np.isnan(got[0]).all()  # NaN * 0 in every sum of that row
        got, want = got[1:], want[1:]
    np.testing.assert_array_equal(got, want)


def test_scales_at_both_ends(gpu):
    """Scale bytes 0 and 252 against their inverses: products near 1 come out whole."""
    import nvfp4_block_scaled_swiglu_amd as nv
    x = np.full((20, 64), 0x7E80, np.uint16)    # 2^126: byte 251, code 4
    x[:, 32:] = 0x0080                          # 2^-126: byte 0, code 2
    w = np.full((40, 64), 0x0100, np.uint16)    # 2^-125: byte 0, code 4
    w[:, 32:] = 0x7E00                          # 2^125
    a = nv.mxfp4_quantize(parity.to_device_bf16(x, gpu))
    b = nv.mxfp4_quantize(parity.to_device_bf16(w, gpu))
    got = nv.mxfp4_gemm_bf16out(a, b).double().cpu().numpy()
    np.testing.assert_array_equal(got, mx_ref.product(mx_ref.round_trip(x), mx_ref.round_trip(w))[0])


def test_no_rows_and_refusals(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    w, _ = operand(24, 64, 1, gpu)
    a = nv.mxfp4_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device=gpu))
    assert nv.mxfp4_gemm_bf16out(a, w).shape == (0, 24)
    b, _ = operand(4, 96, 2, gpu)
    with pytest.raises(ValueError):
        nv.mxfp4_gemm_bf16out(b, w)
    with pytest.raises(ValueError):
        nv.mxfp4_gemm_bf16out(w, w, out=torch.empty(24, 23, dtype=torch.bfloat16, device=gpu))
    with pytest.raises(ValueError):
        nv.mxfp4_gemm_bf16out(nv.Mxfp4Tensor(w.qdata, w.scales, 25, 64), w)
