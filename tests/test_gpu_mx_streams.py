"""GPU: outputs and workspaces that the caller passes to the MXFP4 operators together with a stream
of its own: torch must not give their memory away before that stream is done with them."""
import pytest

from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


def calls(gpu):
    """name -> (caller's tensors, call with a stream) of every entry point that takes an output."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    x = torch.randn(40, 256, device=gpu).bfloat16()
    t = nv.mxfp4_quantize(x)
    c = Case(gpu, [(1, 3000)], group=4).fill(gpu)
    batch = (c.table, c.seq, c.cu)

    def packed(call):
        out = nv.empty_mxfp4(40, 256, gpu)
        return [out.qdata, out.scales], lambda s: call(out=out, stream=s)

    def plain(shape, call):
        out = torch.empty(shape, dtype=torch.bfloat16, device=gpu)
        return [out], lambda s: call(out=out, stream=s)

    def read():
        out = [torch.empty(1, c.kv_heads, c.dim, dtype=torch.bfloat16, device=gpu) for _ in range(2)]
        return out, lambda s: nv.mxfp4_cache_read(c.cache, *batch, 1, out=tuple(out), stream=s)

    def attend():
        size = nv.mxfp4_attention_workspace_bytes(c.cache, *batch, 1, c.heads, 3000)
        assert size > 0
        ws = torch.empty(size, dtype=torch.uint8, device=gpu)
        out = torch.empty_like(c.q)
        return [out, ws], lambda s: nv.mxfp4_attention(c.q, c.cache, *batch, max_kv=3000, out=out, workspace=ws, stream=s)

    return {"quantize": packed(lambda **kw: nv.mxfp4_quantize(x, **kw)),
            "swiglu": packed(lambda **kw: nv.mxfp4_quantize_swiglu(x, x, **kw)),
            "dequantize": plain((40, 256), lambda **kw: nv.mxfp4_dequantize(t, **kw)),
            "gemm": plain((40, 40), lambda **kw: nv.mxfp4_gemm_bf16out(t, t, **kw)),
            "read": read(), "attend": attend()}


@pytest.mark.parametrize("name", ["quantize", "swiglu", "dequantize", "gemm", "read", "attend"])
def test_passed_tensors_are_marked(gpu, monkeypatch, name):
    """Each on the other stream, and none on the current one."""
    import torch
    tensors, call = calls(gpu)[name]
    marked = []
    real = torch.Tensor.record_stream

    def record(self, stream):
        marked.append((self.data_ptr(), stream))
        return real(self, stream)

    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    call(torch.cuda.current_stream())
    assert not marked
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    for t in tensors:
        assert (t.data_ptr(), side) in marked


def test_dropped_tensors_stay_until_the_stream_is_done(gpu):
    """A workspace and an output dropped while the other stream has yet to run the call: their
    blocks are not handed out again meanwhile, and are afterwards."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(1, 3000)], group=4).fill(gpu)
    args = (c.q, c.cache, c.table, c.seq, c.cu)
    size = nv.mxfp4_attention_workspace_bytes(*args[1:], 1, c.heads, 3000)
    want = nv.mxfp4_attention(*args, max_kv=3000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # a size of its own, so that the next request of it would take exactly this block
    ws = torch.empty(size + (37 << 20), dtype=torch.uint8, device=gpu)
    out = torch.empty_like(c.q)
    at = ws.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
    nv.mxfp4_attention(*args, max_kv=3000, out=out, workspace=ws, stream=side)
    n = ws.numel()
    del ws
    held = torch.empty(n, dtype=torch.uint8, device=gpu)
    assert not side.query()  # it had not run yet
    assert held.data_ptr() != at
    held.fill_(0xFF)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
