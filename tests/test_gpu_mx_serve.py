"""GPU: norms and rotation, cache, pages and attention together, as a server uses them: a prompt, answers
forked from it, their tokens one by one, sequences that end, pages that move; eager, in a graph, on
other streams."""
import numpy as np
import pytest

from tests import mx_ref, mx_seq_ref as ref, parity

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, DIM, PAGE, SLOTS, EPS = 6, 2, 64, 16, 5, 1e-6


class Server:
    """The library's side of it, and per slot the keys and values that it must hold (float64)."""

    def __init__(self, gpu, pages=64, seed=0):
        import torch
        import nvfp4_block_scaled_swiglu_amd as nv
        self.gpu, self.nv, self.torch = gpu, nv, torch
        self.rng = np.random.default_rng(seed)
        self.pages = nv.empty_mxfp4_pages(SLOTS, 12, pages, PAGE, gpu)
        self.cache = nv.empty_mxfp4_cache(pages, PAGE, KV_HEADS, DIM, gpu)
        self.rot = nv.mxfp4_rotation(32, gpu, theta=500.0)
        self.w = [mx_ref.f64_to_bits(1 + 0.2 * self.rng.standard_normal(DIM)) for _ in range(2)]
        self.wd = [parity.to_device_bf16(w, gpu) for w in self.w]
        self.held = [([], []) for _ in range(SLOTS)]

    def ints(self, x):
        return self.torch.tensor(x, dtype=self.torch.int32, device=self.gpu)

    def reserve(self, slots, lens):
        done, src, dst = self.nv.mxfp4_pages_reserve(self.pages, self.ints(slots), self.ints(lens))
        assert done.tolist() == [1] * len(slots)
        self.nv.mxfp4_cache_copy(self.cache, src, dst)

    def tokens(self, slots, counts, attend):
        """New tokens for the slots (a run of them: rows of the table), checked."""
        nv, first = self.nv, slots[0]
        assert list(slots) == list(range(first, first + len(slots)))
        n = sum(counts)
        bits = mx_ref.f64_to_bits(self.rng.standard_normal((n, HEADS + 2 * KV_HEADS, DIM)))
        x = parity.to_device_bf16(bits, self.gpu)
        rows = slice(first, first + len(slots))
        batch = (self.pages.block_table[rows], self.pages.seq_lens[rows], self.ints(np.cumsum([0] + list(counts))))
        q = nv.mxfp4_norm_rope_append(self.cache, x[:, :HEADS], x[:, HEADS:-KV_HEADS], x[:, -KV_HEADS:], *batch, self.rot,
                                      q_weight=self.wd[0], k_weight=self.wd[1], eps=EPS)
        out = attend(q, batch)
        freqs, at = self.rot.freqs.cpu().numpy(), 0
        got_q, got = (t.double().cpu() for t in (q, out))
        for s, c in zip(slots, counts):
            keys, values = self.held[s]
            pos = np.arange(len(keys), len(keys) + c)[:, None]
            angle = ref.turns(pos, freqs)
            b = mx_ref.bits_to_f64(bits[at:at + c])
            want, size = ref.norm_rope(b[:, :HEADS], angle, False, EPS, mx_ref.bits_to_f64(self.w[0]))
            assert (np.abs(got_q[at:at + c].numpy() - want) <= ref.norm_rope_tolerance(want, size)).all()
            k, _ = ref.norm_rope(b[:, HEADS:-KV_HEADS], angle, False, EPS, mx_ref.bits_to_f64(self.w[1]))
            keys.extend(mx_ref.round_trip(mx_ref.f64_to_bits(k)))
            values.extend(mx_ref.round_trip(bits[at:at + c, -KV_HEADS:]))
            o, tol = mx_ref.attention(got_q[at:at + c], *(self.torch.from_numpy(np.stack(t)) for t in (keys, values)), DIM ** -0.5)
            assert bool(((got[at:at + c] - o).abs() <= tol).all()), (s, len(keys))
            at += c

    def plain(self, q, batch):
        return self.nv.mxfp4_attention(q, self.cache, *batch)

    def behind(self, table, length):
        """Attention of sequences that all begin with the tokens of a table's row."""
        def attend(q, batch):
            n = batch[1].shape[0]
            return self.nv.mxfp4_attention_prefix(q, self.cache, *batch, table, self.ints([length]), self.ints([0, n]))
        return attend


@pytest.mark.parametrize("prompt", [70, 64, 33, 130])
def test_answers_to_a_prompt(gpu, prompt):
    s = Server(gpu, seed=prompt)
    nv, pages = s.nv, s.pages
    s.reserve([0], [prompt])
    s.tokens([0], [prompt], s.plain)
    assert nv.mxfp4_pages_fork(pages, s.ints([0, 0, 0]), s.ints([1, 2, 3])).tolist() == [1, 1, 1]
    for i in (1, 2, 3):
        s.held[i] = tuple(list(t) for t in s.held[0])
    full = prompt // PAGE * PAGE
    table = pages.block_table[:1].clone()
    table[:, prompt // PAGE:] = -1
    for step in range(6):
        s.reserve([0, 1, 2, 3], [prompt + step + 1] * 4)
        s.tokens([0, 1, 2, 3], [1] * 4, s.behind(table, full))
    # one ends, another is forked in its place, drafts of different lengths, one is cut back
    nv.mxfp4_pages_free(pages, s.ints([2]))
    nv.mxfp4_pages_fork(pages, s.ints([1]), s.ints([2]))
    s.held[2] = tuple(list(t) for t in s.held[1])
    s.reserve([2, 0, 1, 3], [prompt + 6 + n for n in (4, 2, 1, 5)])
    s.tokens([0, 1, 2, 3], [2, 1, 4, 5], s.behind(table, full))
    nv.mxfp4_pages_free(pages, s.ints([3]), s.ints([prompt + 7]))
    s.held[3] = tuple(t[:prompt + 7] for t in s.held[3])
    # the first leaves, pages move to the front, the others go on, behind the table that moved with them
    nv.mxfp4_pages_free(pages, s.ints([0]))
    s.held[0] = ([], [])
    after, src, dst, used = nv.mxfp4_pages_compact(pages)
    nv.mxfp4_cache_copy(s.cache, src, dst)
    s.pages = pages = after
    assert int(used) == int((pages.refs > 0).sum()) and bool((pages.refs[:int(used)] > 0).all())
    table = pages.block_table[1:2].clone()
    lens = [len(s.held[i][0]) for i in (1, 2, 3)]
    for step in range(3):
        s.reserve([1, 2, 3], [n + step + 1 for n in lens])
        s.tokens([1, 2, 3], [1] * 3, s.behind(table, full))
    # a call without rows
    none = s.torch.empty(0, HEADS, DIM, dtype=s.torch.bfloat16, device=gpu)
    batch = (pages.block_table[:1], pages.seq_lens[:1], s.ints([0, 0]))
    q = nv.mxfp4_norm_rope_append(s.cache, none, none[:, :KV_HEADS], none[:, :KV_HEADS], *batch, s.rot, eps=EPS)
    assert s.behind(table, full)(q, batch).shape == none.shape


def state(s):
    return [t.clone() for t in (s.pages.block_table, s.pages.seq_lens, s.pages.refs, s.cache.k_codes, s.cache.k_scales,
                                s.cache.v_codes, s.cache.v_scales)]


def restore(s, saved):
    for t, w in zip((s.pages.block_table, s.pages.seq_lens, s.pages.refs, s.cache.k_codes, s.cache.k_scales, s.cache.v_codes,
                     s.cache.v_scales), saved):
        t.copy_(w)


def step_of(s, slots, x, table, length):
    """One token for each slot, as a function without the host in it: what a graph captures."""
    torch, nv = s.torch, s.nv
    listed, cu, prefix, starts = s.ints(slots), s.ints(list(range(len(slots) + 1))), s.ints([length]), s.ints([0, len(slots)])
    rows = slice(slots[0], slots[-1] + 1)

    def step(stream=None):
        lens = s.pages.seq_lens[rows] + 1
        done, src, dst = nv.mxfp4_pages_reserve(s.pages, listed, lens, stream=stream)
        nv.mxfp4_cache_copy(s.cache, src, dst, stream=stream)
        batch = (s.pages.block_table[rows], s.pages.seq_lens[rows], cu)
        q = nv.mxfp4_norm_rope_append(s.cache, x[:, :HEADS], x[:, HEADS:-KV_HEADS], x[:, -KV_HEADS:], *batch, s.rot,
                                      q_weight=s.wd[0], k_weight=s.wd[1], eps=EPS, stream=stream)
        return [done, src, dst, q, nv.mxfp4_attention_prefix(q, s.cache, *batch, table, prefix, starts, stream=stream)]

    return step


def begun(gpu, seed=0):
    s = Server(gpu, seed=seed)
    s.reserve([0], [70])
    s.tokens([0], [70], s.plain)
    s.nv.mxfp4_pages_fork(s.pages, s.ints([0, 0, 0]), s.ints([1, 2, 3]))
    x = s.torch.randn(4, HEADS + 2 * KV_HEADS, DIM, device=gpu).bfloat16()
    return s, x, step_of(s, [0, 1, 2, 3], x, s.pages.block_table[:1].clone(), 64)


def test_graph(gpu):
    """Two servers' steps captured, replayed with new tokens between eager work; each replay equal to
    the eager step from the same state, the pages and the cache with it."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    nv.nvfp4_init()
    made = [begun(gpu, seed) for seed in (1, 2)]
    graphs, outs = [], []
    for s, x, step in made:
        saved = state(s)
        step()
        torch.cuda.synchronize()
        restore(s, saved)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
        restore(s, saved)
    for i in range(6):
        for (s, x, step), g, out in zip(made, graphs, outs):
            x.copy_(torch.randn(x.shape, device=gpu))
            saved = state(s)
            want = [t.clone() for t in step()]
            after = state(s)
            restore(s, saved)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), i
            for a, b in zip(state(s), after):
                assert torch.equal(a, b), i
            assert out[0].tolist() == [1] * 4


def test_graphs_at_once(gpu):
    """Both graphs replayed at once on two streams: their workspaces are their own."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    nv.nvfp4_init()
    made, graphs, outs, streams = [begun(gpu, seed) for seed in (3, 4)], [], [], [torch.cuda.Stream() for _ in range(2)]
    for s, x, step in made:
        saved = state(s)
        step()
        torch.cuda.synchronize()
        restore(s, saved)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
        restore(s, saved)
    for _ in range(4):
        saved = [state(s) for s, _, _ in made]
        want = [[t.clone() for t in step()] for _, _, step in made]
        for (s, _, _), w in zip(made, saved):
            restore(s, w)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for out, w in zip(outs, want):
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_other_stream(gpu):
    """On a stream given to every call, equal to the current one's results; passed outputs and workspaces
    are marked as used by it."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    s, x, step = begun(gpu, 5)
    saved = state(s)
    want = [t.clone() for t in step()]
    restore(s, saved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens = s.pages.seq_lens[:4] + 1
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(lens, s.pages.seq_lens[:4])


def test_passed_tensors_are_marked(gpu, monkeypatch):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    s, x, _ = begun(gpu, 6)
    batch = (s.pages.block_table[:4], s.pages.seq_lens[:4], s.ints([0, 1, 2, 3, 4]))
    prefix = (s.pages.block_table[:1], s.ints([64]), s.ints([0, 4]))
    q = x[:, :HEADS].contiguous()
    listed, lens = s.ints([0, 1]), s.ints([71, 72])
    pos = s.ints([1, 2, 3, 4])

    def workspace(size):
        return torch.empty(max(size, 16), dtype=torch.uint8, device=gpu)

    ws = [workspace(nv.mxfp4_attention_prefix_workspace_bytes(s.cache, *batch, *prefix, 4, HEADS)),
          workspace(nv.mxfp4_pages_reserve_workspace_bytes(s.pages, 2)), workspace(nv.mxfp4_pages_compact_workspace_bytes(s.pages))]
    outs = [torch.empty_like(q) for _ in range(3)]
    fresh = nv.Mxfp4Pages(torch.empty_like(s.pages.block_table), s.pages.seq_lens, torch.empty_like(s.pages.refs), PAGE)
    calls = [
        ([outs[0], pos, s.rot.freqs, s.wd[0]], lambda st: nv.mxfp4_norm_rope(q, s.rot, pos, weight=s.wd[0], eps=EPS, out=outs[0], stream=st)),
        ([outs[1], s.wd[1]], lambda st: nv.mxfp4_norm_rope_append(s.cache, q, x[:, HEADS:-KV_HEADS], x[:, -KV_HEADS:], *batch, s.rot,
                                                                  k_weight=s.wd[1], eps=EPS, out=outs[1], stream=st)),
        ([outs[2], ws[0], prefix[1]], lambda st: nv.mxfp4_attention_prefix(q, s.cache, *batch, *prefix, out=outs[2], workspace=ws[0], stream=st)),
        ([ws[1], listed, lens, s.pages.refs], lambda st: nv.mxfp4_pages_reserve(s.pages, listed, lens, workspace=ws[1], stream=st)),
        ([ws[2], fresh.refs, fresh.block_table], lambda st: nv.mxfp4_pages_compact(s.pages, out=fresh, workspace=ws[2], stream=st)),
        ([listed, s.pages.seq_lens], lambda st: nv.mxfp4_pages_free(s.pages, listed, stream=st)),
        ([listed, lens], lambda st: nv.mxfp4_pages_fork(s.pages, listed, lens, stream=st)),
        ([s.cache.k_codes, listed], lambda st: nv.mxfp4_cache_copy(s.cache, listed, listed, stream=st)),
    ]
    marked, real = [], torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, st: (marked.append((self.data_ptr(), st)), real(self, st))[1])
    side = torch.cuda.Stream()
    for tensors, call in calls:
        call(torch.cuda.current_stream())
        assert not marked
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        torch.cuda.synchronize()
        for t in tensors:
            assert (t.data_ptr(), side) in marked
        marked.clear()


def test_failures_leave_everything(gpu):
    """Refused calls raise (strict) or return None, count, and write nothing."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    s, x, _ = begun(gpu, 7)
    saved = state(s)
    batch = (s.pages.block_table[:4], s.pages.seq_lens[:4], s.ints([0, 1, 2, 3, 4]))
    small = torch.empty(16, dtype=torch.uint8, device=gpu)
    bad = nv.Mxfp4Pages(s.pages.block_table, s.pages.seq_lens, s.pages.refs, 24)
    calls = {"mxfp4_pages_reserve": lambda **kw: nv.mxfp4_pages_reserve(s.pages, s.ints([0]), s.ints([80]), workspace=small, **kw),
             "mxfp4_pages_compact": lambda **kw: nv.mxfp4_pages_compact(s.pages, out=s.pages, workspace=small, **kw),
             "mxfp4_pages_free": lambda **kw: nv.mxfp4_pages_free(bad, s.ints([0]), **kw),
             "mxfp4_pages_fork": lambda **kw: nv.mxfp4_pages_fork(bad, s.ints([0]), s.ints([4]), **kw),
             "mxfp4_norm_rope_append": lambda **kw: nv.mxfp4_norm_rope_append(
                 s.cache, x[:, :HEADS], x[:, HEADS:-KV_HEADS], x[:, -KV_HEADS:], *batch, eps=-1.0, **kw),
             "mxfp4_norm_rope": lambda **kw: nv.mxfp4_norm_rope(x, eps=0.0, **kw),
             "mxfp4_attention_prefix": lambda **kw: nv.mxfp4_attention_prefix(
                 x[:, :HEADS], s.cache, *batch, s.pages.block_table[:1], s.ints([64]), s.ints([0, 4]), scale=-1.0, **kw)}
    for name, call in calls.items():
        with pytest.raises(nv.Nvfp4Error):
            call(strict=True)
        before = nv.dispatch_counters()[name]["fallbacks"]
        assert call(strict=False) is None
        assert nv.dispatch_counters()[name]["fallbacks"] == before + 1
    with pytest.raises(ValueError):
        nv.mxfp4_cache_copy(s.cache, s.ints([0]), s.ints([1, 2]))
    for a, b in zip(state(s), saved):
        assert torch.equal(a, b)
