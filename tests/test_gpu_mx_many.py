"""GPU: MXFP4 attention of 2^24 rows x heads, 64 heads of 64 over 8."""
import pytest

from tests import mx_ref, parity

pytestmark = pytest.mark.gpu

ROWS, HEADS, KV_HEADS, DIM, PAGE = 1 << 18, 64, 8, 64, 16


def caches(gpu, k, v, table, seq, cu):
    import nvfp4_block_scaled_swiglu_amd as nv
    cache = nv.empty_mxfp4_cache(int(table.max()) + 1, PAGE, KV_HEADS, DIM, gpu)
    nv.mxfp4_cache_append(cache, k, v, table, seq, cu)
    return cache


def test_one_long_prompt(gpu):
    """262,144 rows of one sequence under a window of 40: rows from everywhere against float64."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.arange(ROWS // PAGE, dtype=torch.int32, device=gpu).flip(0)[None]
    seq = torch.tensor([ROWS], dtype=torch.int32, device=gpu)
    cu = torch.tensor([0, ROWS], dtype=torch.int32, device=gpu)
    k, v = (torch.randn(ROWS, KV_HEADS, DIM, generator=g, device=gpu).bfloat16() for _ in range(2))
    q = torch.empty(ROWS, HEADS, DIM, dtype=torch.bfloat16, device=gpu).normal_(generator=g)
    out = nv.mxfp4_attention(q, caches(gpu, k, v, table, seq, cu), table, seq, cu, max_kv=ROWS, window=40)
    for end in (1, 30, 129, 77777, 131073, ROWS - 5, ROWS):
        first = max(0, end - 44)  # rows end - 4 .. end - 1 see tokens from end - 43 on
        n = min(4, end)
        kk, vv = (torch.from_numpy(mx_ref.round_trip(parity.tensor_bits(t[first:end]))) for t in (k, v))
        ref, tol = mx_ref.attention(q[end - n:end].double().cpu(), kk, vv, DIM ** -0.5, window=40)
        assert bool(((out[end - n:end].double().cpu() - ref).abs() <= tol).all()), end


def test_many_sequences(gpu):
    """262,144 sequences of one token each: the output is the token's value."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randperm(ROWS, generator=g, device=gpu).to(torch.int32)[:, None]
    seq = torch.ones(ROWS, dtype=torch.int32, device=gpu)
    cu = torch.arange(ROWS + 1, dtype=torch.int32, device=gpu)
    k, v = (torch.randn(ROWS, KV_HEADS, DIM, generator=g, device=gpu).bfloat16() for _ in range(2))
    q = torch.empty(ROWS, HEADS, DIM, dtype=torch.bfloat16, device=gpu).normal_(generator=g)
    cache = caches(gpu, k, v, table, seq, cu)
    out = nv.mxfp4_attention(q, cache, table, seq, cu)
    want = nv.mxfp4_cache_read(cache, table, seq, cu, ROWS)[1]
    assert torch.equal(out, want.repeat_interleave(HEADS // KV_HEADS, 1))


def test_one_token_of_heads_first_tensors(gpu):
    """Query and output as one token of [heads, tokens, dim] tensors; the others stay as they were."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    from tests.test_gpu_mx_attention import Case
    c = Case(gpu, [(1, 70)], group=4).fill(gpu)
    q, out = (torch.full((c.heads, 9, c.dim), 7.0, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    q[:, 5:6] = c.q.transpose(0, 1)
    got = nv.mxfp4_attention(q.transpose(0, 1)[5:6], c.cache, c.table, c.seq, c.cu, out=out.transpose(0, 1)[3:4])
    c.check(got)
    out[:, 3] = 7.0
    assert (out == 7.0).all()
