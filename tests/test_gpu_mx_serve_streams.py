"""GPU: a decoding step on a stream of its own, everything that it works out among its work there."""
import pytest

from tests.test_gpu_mx_serve import EPS, HEADS, KV_HEADS, begun, restore, state

pytestmark = pytest.mark.gpu


def step_on(s, x, table, length, stream):
    """One token for each of the first four slots. The lengths asked for are worked out on the stream that
    the calls run on, behind what it has to do before."""
    torch, nv = s.torch, s.nv
    listed, cu, prefix, starts = s.ints([0, 1, 2, 3]), s.ints([0, 1, 2, 3, 4]), s.ints([length]), s.ints([0, 4])
    side = stream is not None
    given = stream if side else torch.cuda.current_stream()
    given.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(given):
        if side:
            torch.cuda._sleep(2000000)  # about a millisecond, before the lengths are read
        lens = s.pages.seq_lens[:4] + 1
    done, src, dst = nv.mxfp4_pages_reserve(s.pages, listed, lens, stream=stream)
    nv.mxfp4_cache_copy(s.cache, src, dst, stream=stream)
    batch = (s.pages.block_table[:4], s.pages.seq_lens[:4], cu)
    q = nv.mxfp4_norm_rope_append(s.cache, x[:, :HEADS], x[:, HEADS:-KV_HEADS], x[:, -KV_HEADS:], *batch, s.rot,
                                  q_weight=s.wd[0], k_weight=s.wd[1], eps=EPS, stream=stream)
    out = nv.mxfp4_attention_prefix(q, s.cache, *batch, table, prefix, starts, stream=stream)
    torch.cuda.current_stream().wait_stream(given)
    return [lens, done, src, dst, q, out]


def test_steps_on_another_stream(gpu):
    """Three steps, each equal to the one on the current stream from the same state: outputs, pages and cache."""
    import torch
    s, x, _ = begun(gpu, 8)
    table = s.pages.block_table[:1].clone()
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(torch.randn(x.shape, device=gpu))
        saved = state(s)
        want = [t.clone() for t in step_on(s, x, table, 64, None)]
        after = state(s)
        restore(s, saved)
        got = step_on(s, x, table, 64, side)
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
        for a, b in zip(state(s), after):
            assert torch.equal(a, b), i
        assert got[1].tolist() == [1] * 4 and got[0].tolist() == [71 + i] * 4
