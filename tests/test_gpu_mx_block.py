"""GPU: the MXFP4 operators together, as a transformer block uses them - QKV projection, cache
append, attention, output projection, SwiGLU MLP - on other streams and in a HIP graph."""
import numpy as np
import pytest

from tests import mx_ref, parity

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS, DIM, MLP, PAGE = 256, 6, 2, 64, 320, 16
LENS = [(1, 70), (9, 9), (3, 40)]


class Block:
    def __init__(self, gpu, seed=0):
        import torch
        import nvfp4_block_scaled_swiglu_amd as nv
        rng = np.random.default_rng(seed)
        self.bits = {n: mx_ref.f64_to_bits(rng.standard_normal(s) * 0.05) for n, s in
                     dict(qkv=((HEADS + 2 * KV_HEADS) * DIM, HIDDEN), out=(HIDDEN, HEADS * DIM), fc1=(2 * MLP, HIDDEN),
                          fc2=(HIDDEN, MLP)).items()}
        self.w = {n: nv.mxfp4_quantize(parity.to_device_bf16(b, gpu)) for n, b in self.bits.items()}
        self.tokens = sum(q for q, _ in LENS)
        pages = [-(-kv // PAGE) for _, kv in LENS]
        self.table = torch.full((len(LENS), max(pages)), -1, dtype=torch.int32, device=gpu)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = torch.arange(at, at + n, dtype=torch.int32)
            at += n
        self.seq = torch.tensor([kv for _, kv in LENS], dtype=torch.int32, device=gpu)
        self.cu = torch.tensor(np.cumsum([0] + [q for q, _ in LENS]), dtype=torch.int32, device=gpu)
        old = torch.tensor([kv - q for q, kv in LENS], dtype=torch.int32, device=gpu)
        self.cache = nv.empty_mxfp4_cache(at, PAGE, KV_HEADS, DIM, gpu)
        self.old_bits = [mx_ref.f64_to_bits(rng.standard_normal((sum(kv - q for q, kv in LENS), KV_HEADS, DIM)))
                         for _ in range(2)]
        old_cu = torch.tensor(np.cumsum([0] + [kv - q for q, kv in LENS]), dtype=torch.int32, device=gpu)
        nv.mxfp4_cache_append(self.cache, *(parity.to_device_bf16(b, gpu) for b in self.old_bits), self.table, old, old_cu)

    def forward(self, x, stream=None):
        import nvfp4_block_scaled_swiglu_amd as nv
        kw = dict(stream=stream)
        qkv = nv.mxfp4_gemm_bf16out(nv.mxfp4_quantize(x, **kw), self.w["qkv"], **kw).view(self.tokens, -1, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        nv.mxfp4_cache_append(self.cache, k, v, self.table, self.seq, self.cu, **kw)
        o = nv.mxfp4_attention(q, self.cache, self.table, self.seq, self.cu, max_kv=70, **kw)
        y = nv.mxfp4_gemm_bf16out(nv.mxfp4_quantize(o.view(self.tokens, -1), **kw), self.w["out"], **kw)
        gu = nv.mxfp4_gemm_bf16out(nv.mxfp4_quantize(y, **kw), self.w["fc1"], **kw)
        act = nv.mxfp4_quantize_swiglu(gu[:, :MLP], gu[:, MLP:], **kw)
        return dict(qkv=qkv, o=o, y=y, gu=gu, z=nv.mxfp4_gemm_bf16out(act, self.w["fc2"], **kw))


def inputs(tokens, seed):
    return mx_ref.f64_to_bits(np.random.default_rng(seed).standard_normal((tokens, HIDDEN)))


def test_every_stage_against_the_definitions(gpu):
    """Each stage from the bytes that the stage before gave, so that one stage's rounding is not
    another's error."""
    import torch
    import oracle
    b = Block(gpu)
    xb = inputs(b.tokens, 1)
    got = b.forward(parity.to_device_bf16(xb, gpu))
    bits = {n: parity.tensor_bits(t.contiguous()) for n, t in got.items()}

    def product(name, x, n, k):
        ref, mags = mx_ref.product(mx_ref.round_trip(x), mx_ref.round_trip(b.bits[n]))
        off = np.abs(mx_ref.bits_to_f64(bits[name]).reshape(ref.shape) - ref)
        assert (off <= mx_ref.product_tolerance(ref, mags, k)).all(), name

    product("qkv", xb, "qkv", HIDDEN)
    product("y", bits["o"].reshape(b.tokens, -1), "out", HEADS * DIM)
    product("gu", bits["y"], "fc1", HIDDEN)
    gate, up = bits["gu"][:, :MLP], bits["gu"][:, MLP:]
    silu = oracle.silu_table()[gate]
    product("z", mx_ref.f64_to_bits(mx_ref.bits_to_f64(silu) * mx_ref.bits_to_f64(up)), "fc2", MLP)
    new = bits["qkv"].reshape(b.tokens, -1, DIM)
    row = old = 0
    for q, kv in LENS:
        kvs = [np.concatenate([mx_ref.round_trip(b.old_bits[j][old:old + kv - q]),
                               mx_ref.round_trip(new[row:row + q, HEADS + j * KV_HEADS:HEADS + (j + 1) * KV_HEADS])])
               for j in range(2)]
        ref, tol = mx_ref.attention(torch.from_numpy(mx_ref.bits_to_f64(new[row:row + q, :HEADS])),
                                    *(torch.from_numpy(t) for t in kvs), DIM ** -0.5)
        off = (torch.from_numpy(mx_ref.bits_to_f64(bits["o"][row:row + q])) - ref).abs()
        assert bool((off <= tol).all())
        row, old = row + q, old + kv - q


def test_other_stream(gpu):
    """On a stream of its own, with inputs made on the default stream and waited for, twice."""
    import torch
    b = Block(gpu)
    x = parity.to_device_bf16(inputs(b.tokens, 2), gpu)
    want = b.forward(x)
    side = torch.cuda.Stream()
    for _ in range(2):
        side.wait_stream(torch.cuda.current_stream())
        got = b.forward(x.clone(), stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_graph(gpu):
    """Captured once, replayed with new inputs between eager calls, each replay equal to the eager
    result; a second captured block shares nothing with the first."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    nv.nvfp4_init()
    blocks = [Block(gpu, s) for s in (0, 1)]
    xs = [parity.to_device_bf16(inputs(b.tokens, 3), gpu) for b in blocks]
    for b, x in zip(blocks, xs):
        b.forward(x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b, x in zip(blocks, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.forward(x))
        graphs.append(g)
    for seed in (10, 11, 12):
        for b, x, g, out in zip(blocks, xs, graphs, outs):
            x.copy_(parity.to_device_bf16(inputs(b.tokens, seed), gpu))
            g.replay()
            got = {n: t.clone() for n, t in out.items()}
            want = b.forward(x)
            torch.cuda.synchronize()
            for n in want:
                assert torch.equal(got[n], want[n]), (seed, n)


def test_graph_of_split_attention(gpu):
    """Two captured calls that need workspaces, replayed at once on two streams."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    nv.nvfp4_init()
    g = torch.Generator(device="cuda").manual_seed(5)
    kv, page = 6000, 64
    pages = -(-kv // page)
    cache = nv.empty_mxfp4_cache(pages, page, 2, 128, gpu)
    table = torch.randperm(pages, generator=g, device=gpu).to(torch.int32)[None]
    seq = torch.tensor([kv], dtype=torch.int32, device=gpu)
    cu = torch.tensor([0, kv], dtype=torch.int32, device=gpu)
    k, v = (torch.randn(kv, 2, 128, generator=g, device=gpu).bfloat16() for _ in range(2))
    nv.mxfp4_cache_append(cache, k, v, table, seq, cu)
    one = torch.tensor([0, 1], dtype=torch.int32, device=gpu)
    qs = [torch.randn(1, 8, 128, generator=g, device=gpu).bfloat16() for _ in range(2)]
    assert nv.mxfp4_attention_workspace_bytes(cache, table, seq, one, 1, 8, kv) > 0
    want = [nv.mxfp4_attention(q, cache, table, seq, one, max_kv=kv) for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in qs]
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(nv.mxfp4_attention(q, cache, table, seq, one, max_kv=kv))
        graphs.append(graph)
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for out, w in zip(outs, want):
            assert torch.equal(out, w)
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
