"""GPU: forms of the MXFP4 attention's plan that only certain sizes of a batch choose."""
import pytest

from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", [{}, dict(window=150, sinks=20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_few_pieces_of_many_single_tokens(gpu, dim, call):
    """Twenty sequences of 8 kv heads, one of them a prompt, over what may be long caches: single
    tokens in 12 pieces (joined by a wave a row and head), the prompt in 4, 3 and 1."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    lens = [(1, 1 + 23 * i) for i in range(10)] + [(200, 250)] + [(1 + i % 3, 1500 + i) for i in range(9)]
    c = Case(gpu, lens, kv_heads=8, group=4, dim=dim, page=64).fill(gpu)
    args = (c.q, c.cache, c.table, c.seq, c.cu)
    out = nv.mxfp4_attention(*args, max_kv=1 << 13, **call)
    c.check(out, **call)
    for _ in range(3):
        assert torch.equal(out, nv.mxfp4_attention(*args, max_kv=1 << 13, **call))


@pytest.mark.parametrize("rows,kv", [(17, 60), (32, 900), (31, 33)])
def test_two_row_tiles(gpu, rows, kv):
    """17 to 32 rows of heads of 64: two row tiles of the few-rows form, whole and in pieces."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(rows, kv), (rows, kv + 7)], group=1, dim=64).fill(gpu)
    for max_kv in (1, 1 << 11, 1 << 14):
        for call in ({}, dict(causal=False), dict(window=20, sinks=3)):
            c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=max_kv, **call), **call)
