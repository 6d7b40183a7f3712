"""GPU: the MXFP4 operators where offsets pass 32 bits."""
import pytest

from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 64])
def test_far_pages(gpu, page):
    """A cache whose codes take more than 4 GiB each of K and V, with the batch's pages at its end."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    from tests import parity
    c = Case(gpu, [(1, 200), (1, 77)], group=4, page=page)
    prompt = Case(gpu, [(70, 90), (33, 150)], group=2, page=page)
    for case in (c, prompt):
        near = case.cache
        pages = (1 << 32) // (case.kv_heads * page * case.dim // 2) + near.num_pages
        far = nv.empty_mxfp4_cache(pages, page, case.kv_heads, case.dim, gpu)
        assert far.k_codes.numel() > 1 << 32
        shift = pages - near.num_pages
        there = (case.table >= 0) & (case.table < near.num_pages)
        table = torch.where(there, case.table + shift, case.table.clamp(max=-1))
        k, v = parity.to_device_bf16(case.k_bits, gpu), parity.to_device_bf16(case.v_bits, gpu)
        nv.mxfp4_cache_append(far, k, v, table, case.seq, case.all_cu)
        case.fill(gpu)
        for a, b in zip(nv.mxfp4_cache_read(far, table, case.seq, case.all_cu, case.cached),
                        nv.mxfp4_cache_read(near, case.table, case.seq, case.all_cu, case.cached)):
            assert torch.equal(a, b)
        for max_kv in (200, 1 << 14):
            case.check(nv.mxfp4_attention(case.q, far, table, case.seq, case.cu, max_kv=max_kv))
        del far


def test_far_rows_of_a_product(gpu):
    """An output of more than 2^31 elements: rows of A with a single one pick columns of W."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    m, n, k = 70001, 32776, 32
    assert m * n > 1 << 31
    pick = torch.arange(m, device=gpu) % k
    a = torch.zeros(m, k, dtype=torch.bfloat16, device=gpu)
    a[torch.arange(m, device=gpu), pick] = 1.0
    w = torch.randint(-6, 7, (n, k), device=gpu).bfloat16()
    w = torch.where(w.abs() == 5, 4.0, w.float()).bfloat16()
    w[:, 0] = 6.0  # every block's scale is 1
    out = nv.mxfp4_gemm_bf16out(nv.mxfp4_quantize(a), nv.mxfp4_quantize(w))
    for r0, r1 in ((0, 40), (32760, 32800), (65500, 65560), (m - 300, m)):
        assert torch.equal(out[r0:r1], w[:, pick[r0:r1]].t())


def test_far_rows_of_a_quantization(gpu):
    """An input of more than 2^31 elements: the last rows as quantized by themselves, and back."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rows, k, last = 70016, 32768, 128
    assert rows * k > 1 << 31
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device=gpu)
    x[-last:] = torch.randn(last, k, device=gpu).bfloat16()
    t, tail = nv.mxfp4_quantize(x), nv.mxfp4_quantize(x[-last:])
    assert torch.equal(t.qdata[-last:], tail.qdata)
    assert torch.equal(t.scales[-tail.scales.numel():], tail.scales)  # the last tile of 128 rows
    del x
    assert torch.equal(nv.mxfp4_dequantize(t)[-last:], nv.mxfp4_dequantize(tail))
