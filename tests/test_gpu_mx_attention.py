"""GPU: the paged MXFP4 cache and attention over it, against float64 row by row."""
import math

import numpy as np
import pytest

from tests import mx_ref, parity

pytestmark = pytest.mark.gpu


class Case:
    """A ragged batch with its cache: lens is [(new rows, cached tokens)]; garbage everywhere that
    no token lives, page numbers shuffled, unused table entries out of range."""

    def __init__(self, gpu, lens, kv_heads=2, dim=128, page=16, group=1, seed=0, spare=2):
        import torch
        import nvfp4_block_scaled_swiglu_amd as nv
        rng = np.random.default_rng(seed)
        self.lens, self.kv_heads, self.dim, self.page, self.heads = lens, kv_heads, dim, page, kv_heads * group
        pages = [-(-kv // page) for _, kv in lens]
        count = sum(pages) + spare
        most = max(max(pages), 1) + 1
        self.table_np = rng.choice(np.array([-1, count, 2 ** 31 - 1, -2 ** 31]), (len(lens), most)).astype(np.int32)
        order = rng.permutation(count).astype(np.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table_np[i, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.table = torch.from_numpy(self.table_np).to(gpu)
        self.seq = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=gpu)
        self.cu = torch.tensor(np.cumsum([0] + [q for q, _ in lens]), dtype=torch.int32, device=gpu)
        self.all_cu = torch.tensor(np.cumsum([0] + [kv for _, kv in lens]), dtype=torch.int32, device=gpu)
        self.tokens = sum(q for q, _ in lens)
        self.cached = sum(kv for _, kv in lens)
        self.cache = nv.empty_mxfp4_cache(count, page, kv_heads, dim, gpu)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(255)  # NaN wherever nothing is written
        scale = np.exp2(rng.integers(-1, 2, (1, kv_heads, dim // 32))).repeat(32, 2)
        self.k_bits = mx_ref.f64_to_bits(rng.standard_normal((self.cached, kv_heads, dim)) * scale)
        self.v_bits = mx_ref.f64_to_bits(rng.standard_normal((self.cached, kv_heads, dim)) + 0.25)
        self.q_bits = mx_ref.f64_to_bits(rng.standard_normal((self.tokens, self.heads, dim)))
        self.q = parity.to_device_bf16(self.q_bits, gpu)

    def fill(self, gpu):
        import nvfp4_block_scaled_swiglu_amd as nv
        nv.mxfp4_cache_append(self.cache, parity.to_device_bf16(self.k_bits, gpu), parity.to_device_bf16(self.v_bits, gpu),
                              self.table, self.seq, self.all_cu)
        return self

    def check(self, out, scale=None, hidden=None, **kw):
        import torch
        scale = self.dim ** -0.5 if scale is None else scale
        k = torch.from_numpy(mx_ref.round_trip(self.k_bits))
        v = torch.from_numpy(mx_ref.round_trip(self.v_bits))
        q = torch.from_numpy(mx_ref.bits_to_f64(self.q_bits))
        got = out.double().cpu()
        at, base = 0, 0
        for i, (n, kv) in enumerate(self.lens):
            ref, tol = mx_ref.attention(q[at:at + n], k[base:base + kv], v[base:base + kv], scale,
                                        hidden=None if hidden is None else hidden[i], **kw)
            g = got[at:at + n]
            nan = torch.isnan(ref)
            assert torch.equal(torch.isnan(g), nan), (i, int(torch.isnan(g).sum()), int(nan.sum()))
            off = torch.where(nan, 0.0, (g - ref).abs())
            over = (off - torch.where(nan, 1.0, tol)).flatten()
            worst = int(over.argmax()) if over.numel() else 0
            fine = not over.numel() or float(over[worst]) <= 0
            assert fine, (i, worst, float(off.flatten()[worst]), float(tol.flatten()[worst]), float(ref.flatten()[worst]))
            at, base = at + n, base + kv


CACHES = [
    (dict(dim=128, page=16), [(1, 1), (3, 17), (0, 5), (20, 20)]),
    (dict(dim=64, page=32, kv_heads=3), [(33, 64), (2, 31), (65, 65)]),
    (dict(dim=256, page=128, kv_heads=1), [(1, 300), (130, 131)]),
    (dict(dim=128, page=64, kv_heads=8), [(1, n) for n in range(1, 70)]),
]


@pytest.mark.parametrize("kw,lens", CACHES)
def test_append_and_read(gpu, kw, lens):
    """Whole caches written, then the last rows of each overwritten and read back; bytes in the
    pages as the format says, everything else as it was."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, **kw)
    before = [t.clone() for t in (c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales)]
    c.fill(gpu)
    k, v = nv.mxfp4_cache_read(c.cache, c.table, c.seq, c.all_cu, c.cached)
    np.testing.assert_array_equal(k.double().cpu().numpy(), mx_ref.round_trip(c.k_bits))
    np.testing.assert_array_equal(v.double().cpu().numpy(), mx_ref.round_trip(c.v_bits))
    # the bytes, by the layout; slots of no token keep theirs
    want = [b.cpu().numpy().copy() for b in before]
    row = 0
    for i, (_, kv) in enumerate(lens):
        for t in range(kv):
            p, s = c.table_np[i, t // c.page], t % c.page
            for j, b in ((0, c.k_bits), (2, c.v_bits)):
                want[j][p, :, s], want[j + 1][p, :, s] = mx_ref.quantize(b[row])
            row += 1
    for t, w in zip((c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales), want):
        np.testing.assert_array_equal(t.cpu().numpy(), w)
    # the batch's own rows only: new values over the last tokens, strided inputs and outputs
    rng = np.random.default_rng(9)
    new = mx_ref.f64_to_bits(rng.standard_normal((c.tokens, 3 * c.kv_heads, c.dim)))
    packed = parity.to_device_bf16(new, gpu)
    nv.mxfp4_cache_append(c.cache, packed[:, c.kv_heads:2 * c.kv_heads], packed[:, 2 * c.kv_heads:], c.table, c.seq, c.cu)
    hold = torch.full((c.tokens, 2, c.kv_heads, c.dim), 7.0, dtype=torch.bfloat16, device=gpu)
    k, v = nv.mxfp4_cache_read(c.cache, c.table, c.seq, c.cu, c.tokens, out=(hold[:, 0], hold[:, 1]))
    np.testing.assert_array_equal(k.double().cpu().numpy(), mx_ref.round_trip(new[:, c.kv_heads:2 * c.kv_heads]))
    np.testing.assert_array_equal(v.double().cpu().numpy(), mx_ref.round_trip(new[:, 2 * c.kv_heads:]))


def test_rows_without_a_place(gpu):
    """More rows than cached tokens, pages that are not there, rows behind the last sequence: the
    first two are skipped by the append and read as zeros, the last stay as they were."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(40, 40), (20, 20)], page=16)
    c.table[0, 1] = -1
    c.table[1, 0] = c.cache.num_pages
    seq = torch.tensor([35, 20], dtype=torch.int32, device=gpu)
    rows = 64  # four behind the last sequence
    x = torch.ones(rows, c.kv_heads, c.dim, dtype=torch.bfloat16, device=gpu)
    before = c.cache.k_codes.clone()
    nv.mxfp4_cache_append(c.cache, x, x, c.table, seq, c.cu)
    hold = [torch.full_like(x, 7.0) for _ in range(2)]
    k, v = nv.mxfp4_cache_read(c.cache, c.table, seq, c.cu, rows, out=tuple(hold))
    pos = torch.cat([torch.arange(40) - 5, torch.arange(20)])
    there = (pos >= 0) & ~((torch.arange(60) < 40) & (pos // 16 == 1)) & ~((torch.arange(60) >= 40) & (pos < 16))
    want = torch.where(there, 1.0, 0.0)
    for t in (k, v):
        assert torch.equal(t[:60, 0, 0].float().cpu(), want)
        assert (t[60:] == 7.0).all()
    changed = (c.cache.k_codes != before).any(-1).any(1).sum()  # slots written
    assert int(changed) <= int(there.sum())


# (kwargs of Case, lengths, kwargs of attention)
ATTENTION = [
    # single tokens: every group size class, caches of one token, of a tile, around a tile and a page
    (dict(group=1), [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200)], {}),
    (dict(group=7, kv_heads=3, page=64), [(1, 1), (1, 63), (1, 130), (1, 500)], {}),
    (dict(group=16, kv_heads=1, dim=64), [(1, 100), (1, 7)], {}),
    (dict(group=20, kv_heads=2, dim=256, page=32), [(1, 77), (1, 129)], {}),
    (dict(group=40, kv_heads=1), [(1, 90), (1, 33)], {}),
    # several new tokens: rows of a sequence in one wave, then in several workgroups
    (dict(group=4), [(5, 70), (3, 3), (8, 8)], {}),
    (dict(group=3, dim=64), [(21, 100), (64, 64), (1, 40)], {}),
    (dict(group=7, kv_heads=1), [(100, 300), (1, 20), (37, 37)], {}),
    (dict(group=5, kv_heads=1, dim=256, page=64), [(70, 150), (33, 33)], {}),
    # no mask but the lengths
    (dict(group=2), [(9, 40), (1, 100)], dict(causal=False)),
    (dict(group=2, kv_heads=1), [(150, 170)], dict(causal=False)),
    # windows and first tokens, inside a tile, across tiles, larger than the cache, without each other
    (dict(group=4), [(1, 300), (1, 20), (3, 100)], dict(window=40, sinks=5)),
    (dict(group=2, kv_heads=1), [(160, 400), (30, 30)], dict(window=33, sinks=1)),
    (dict(group=2, kv_heads=1, dim=64), [(160, 400), (30, 30)], dict(window=64, sinks=70)),
    (dict(group=1, dim=64), [(70, 200), (2, 199)], dict(window=1)),
    (dict(group=1), [(5, 50)], dict(window=1000, sinks=1000)),
    # a long cache: the work is split and joined
    (dict(group=6, page=32), [(1, 3000), (1, 10), (1, 1500)], {}),
    (dict(group=6, page=256, dim=64), [(4, 5000)], dict(window=2500, sinks=3)),
    (dict(group=6, kv_heads=1, dim=256), [(2, 2000), (1, 65)], {}),
    (dict(group=2, kv_heads=1), [(130, 2500)], {}),
    # rows that see nothing: an empty cache, more rows than tokens
    (dict(group=2), [(3, 0), (1, 5), (0, 9), (2, 0)], {}),
    (dict(group=3, kv_heads=1), [(50, 20), (200, 100)], {}),
]


@pytest.mark.parametrize("kw,lens,call", ATTENTION)
def test_attention(gpu, kw, lens, call):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, **kw).fill(gpu)
    longest = max(1, max(kv for _, kv in lens))
    out = nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=longest, **call)
    c.check(out, **call)
    # the same again, bit for bit; and cut as for a much longer and a shorter cache
    assert torch.equal(out, nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=longest, **call))
    c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=1 << 16, **call), **call)
    c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=1, **call), **call)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 4.0])
def test_scale_and_large_scores(gpu, scale):
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(4, 200), (1, 900)], group=4).fill(gpu)
    c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, scale=scale), scale=scale)


@pytest.mark.parametrize("q,kv", [(1, 700), (80, 300)])
def test_maximum_that_keeps_rising(gpu, q, kv):
    """Keys that grow along the cache raise the running maximum in every tile, falling ones never
    after the first."""
    import nvfp4_block_scaled_swiglu_amd as nv
    for sign in (1, -1):
        c = Case(gpu, [(q, kv)], group=2, kv_heads=1)
        ramp = np.linspace(0.1, 30.0, kv)[::sign, None, None]
        c.k_bits = mx_ref.f64_to_bits(np.abs(mx_ref.bits_to_f64(c.k_bits)) * ramp)
        c.q_bits = c.q_bits & 0x7FFF
        c.q = parity.to_device_bf16(c.q_bits, gpu)
        c.fill(gpu)
        c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, scale=0.05), scale=0.05)


@pytest.mark.parametrize("call", [{}, dict(window=50, sinks=4)])
@pytest.mark.parametrize("kw,lens", [(dict(group=2), [(1, 200), (6, 90)]), (dict(group=4, kv_heads=1), [(100, 160)]),
                                     (dict(group=4, dim=64), [(7, 65)]), (dict(group=1, dim=256), [(40, 70)])])
def test_nan_reaches_the_rows_that_see_it(gpu, kw, lens, call):
    """A NaN block of V makes its 32 elements NaN, one of K whole rows, in the rows that see the
    token and in no others."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, **kw)
    base = 0
    for i, (n, kv) in enumerate(lens):
        c.v_bits[base + kv - 1 - n // 3, 0, 33] = 0x7FC0   # seen by the last rows
        c.v_bits[base + 2, -1, 1] = 0x7F80                 # a first token: hidden where a window has passed it
        if i == 0:
            c.k_bits[base + kv - 2, 0, 0] = 0xFF80
        base += kv
    c.fill(gpu)
    c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, **call), **call)


def test_pages_that_are_not_there(gpu):
    """Tokens on them are not seen; a sequence with nothing but such pages gives zeros."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    lens = [(3, 100), (1, 40), (40, 90)]
    c = Case(gpu, lens, group=3, page=16).fill(gpu)
    hidden = [torch.zeros(kv, dtype=torch.bool) for _, kv in lens]
    for i, p, bad in ((0, 1, -1), (0, 6, c.cache.num_pages), (2, 0, 2 ** 31 - 1), (1, 0, -5), (1, 1, -1), (1, 2, -2 ** 31)):
        c.table[i, p] = bad
        hidden[i][p * 16:(p + 1) * 16] = True
    for kv in (100, 4096):
        out = nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=kv)
        c.check(out, hidden=hidden)
        assert (out[3] == 0).all()


@pytest.mark.parametrize("q,max_kv", [(1, 64), (1, 1 << 16), (30, 64), (30, 1 << 16)])
def test_rows_behind_the_last_sequence(gpu, q, max_kv):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(q, 300), (q, 50)], group=4).fill(gpu)
    x = torch.cat([c.q, torch.full_like(c.q[:1], float("nan")).repeat(5, 1, 1)])
    hold = torch.full_like(x, 7.0)
    out = nv.mxfp4_attention(x, c.cache, c.table, c.seq, c.cu, out=hold, max_kv=max_kv)
    assert out is hold and (out[c.tokens:] == 7.0).all()
    c.check(out)


def test_strided_query_and_output(gpu):
    """q as a slice of a packed projection, out as a slice of a wider tensor and heads-first."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(40, 90), (1, 33)], group=2).fill(gpu)
    packed = torch.zeros(c.tokens, c.heads + 2 * c.kv_heads, c.dim, dtype=torch.bfloat16, device=gpu)
    packed[:, :c.heads] = c.q
    hold = torch.full((c.tokens, c.heads + 1, c.dim), 7.0, dtype=torch.bfloat16, device=gpu)
    c.check(nv.mxfp4_attention(packed[:, :c.heads], c.cache, c.table, c.seq, c.cu, out=hold[:, 1:]))
    assert (hold[:, 0] == 7.0).all()
    first = torch.empty(c.heads, c.tokens, c.dim, dtype=torch.bfloat16, device=gpu)
    c.check(nv.mxfp4_attention(c.q.transpose(0, 1).contiguous().transpose(0, 1), c.cache, c.table, c.seq, c.cu,
                               out=first.transpose(0, 1)))


def test_lengths_out_of_range_are_clamped(gpu):
    """A cached length beyond the block table, below zero, and row starts beyond the tensor."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(2, 48), (2, 32)], group=2).fill(gpu)
    table = c.table[:, :3].contiguous()
    table[1, 2] = -1
    seq = torch.tensor([2 ** 31 - 1, -7], dtype=torch.int32, device=gpu)
    out = nv.mxfp4_attention(c.q, c.cache, table, seq, c.cu)
    want = nv.mxfp4_attention(c.q, c.cache, table, c.seq, c.cu)
    assert torch.equal(out[:2], want[:2]) and (out[2:] == 0).all()
    cu = torch.tensor([0, 2, 2 ** 31 - 1], dtype=torch.int32, device=gpu)
    assert torch.equal(nv.mxfp4_attention(c.q, c.cache, table, c.seq, cu), want)


def test_nothing_to_do(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(1, 5)])
    e = c.q[:0]
    cu = torch.zeros(2, dtype=torch.int32, device=gpu)
    assert nv.mxfp4_attention(e, c.cache, c.table, c.seq, cu).shape == e.shape
    kv = torch.empty(0, c.kv_heads, c.dim, dtype=torch.bfloat16, device=gpu)
    assert nv.mxfp4_cache_append(c.cache, kv, kv, c.table, c.seq, cu) is c.cache
    none = torch.empty(0, 2, dtype=torch.int32, device=gpu)
    hold = torch.full_like(c.q, 7.0)
    nv.mxfp4_attention(c.q, c.cache, none, none[:, 0], cu[:1], out=hold)
    assert (hold == 7.0).all()


def test_refusals(gpu):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(2, 20)], group=2)
    good = (c.cache, c.table, c.seq, c.cu)
    for bad in (dict(q=c.q.float()), dict(q=c.q[:, :, ::2]), dict(q=c.q[:, :, :64])):
        with pytest.raises(ValueError):
            nv.mxfp4_attention(bad["q"], *good)
    with pytest.raises(ValueError):
        nv.mxfp4_attention(c.q, c.cache, c.table.long(), c.seq, c.cu)
    with pytest.raises(ValueError):
        nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu[:1])
    with pytest.raises(ValueError):
        nv.mxfp4_attention(c.q, *good, out=torch.empty_like(c.q[:1]))
    for kw, status in ((dict(window=4, causal=False), 1), (dict(sinks=4), 1), (dict(scale=0.0), 1),
                       (dict(max_kv=1 << 20, workspace=torch.empty(64, dtype=torch.uint8, device=gpu)), 4)):
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.mxfp4_attention(c.q, *good, **kw)
        assert e.value.status == status
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mxfp4_attention(c.q[:, :3], *good)
    assert e.value.status == 1
    assert nv.mxfp4_attention(c.q[:, :3], *good, strict=False) is None
    x = torch.zeros(2, c.kv_heads, c.dim, dtype=torch.bfloat16, device=gpu)
    with pytest.raises(ValueError):
        nv.mxfp4_cache_append(c.cache, x[:, :1], x, c.table, c.seq, c.cu)
    with pytest.raises(nv.Nvfp4Error):
        nv.mxfp4_cache_read(*good, 2, out=(x[:1].expand(2, -1, -1), x))


@pytest.mark.parametrize("call", [{}, dict(window=700, sinks=70), dict(causal=False)])
@pytest.mark.parametrize("kw,lens", [(dict(group=2), [(40, 1500), (33, 80)]), (dict(group=3, kv_heads=1, dim=64), [(50, 1300)]),
                                     (dict(group=1, dim=256, page=32), [(70, 1100), (3, 0), (40, 500)])])
def test_prompts_in_pieces(gpu, kw, lens, call):
    """More rows than the few-rows form takes, over a cache that is split."""
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, **kw).fill(gpu)
    args = (c.cache, c.table, c.seq, c.cu)
    assert nv.mxfp4_attention_workspace_bytes(*args, c.tokens, c.heads, 1 << 14) > 0
    c.check(nv.mxfp4_attention(c.q, *args, max_kv=1 << 14, **call), **call)


@pytest.mark.parametrize("q", [1, 90])
def test_bounds_that_bound_nothing(gpu, q):
    """The largest max_kv, window and sinks are those of no limit."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(q, 300), (q, 91)], group=2).fill(gpu)
    args = (c.q, c.cache, c.table, c.seq, c.cu)
    most = 2 ** 63 - 1
    for kw in (dict(max_kv=most), dict(max_kv=most, window=most, sinks=most), dict(window=most), dict(window=1, sinks=most)):
        c.check(nv.mxfp4_attention(*args, **kw))


@pytest.mark.parametrize("q", [1, 40])
def test_pages_of_two_sequences(gpu, q):
    """Sequences that share the pages of a common beginning, a table that is a slice of a wider
    one, and the queries' own memory as output."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(q, 160), (q, 160)], group=2).fill(gpu)
    wide = torch.full((2, c.table.shape[1] + 3), -1, dtype=torch.int32, device=gpu)
    wide[:, 2:2 + c.table.shape[1]] = c.table
    wide[1, 2:8] = wide[0, 2:8]  # tokens 0 .. 95 of the first
    half = c.k_bits.shape[0] // 2
    for bits in (c.k_bits, c.v_bits):
        bits[half:half + 96] = bits[:96]
    table = wide[:, 2:2 + c.table.shape[1]]
    own = c.q.clone()
    for kv in (160, 1 << 14):
        c.check(nv.mxfp4_attention(c.q, c.cache, table, c.seq, c.cu, max_kv=kv))
    assert nv.mxfp4_attention(own, c.cache, table, c.seq, c.cu, out=own) is own
    c.check(own)


@pytest.mark.parametrize("call", [{}, dict(window=5000, sinks=3), dict(causal=False)])
@pytest.mark.parametrize("kw,lens", [(dict(group=2), [(150, 190), (1, 900), (0, 50), (8, 33), (1, 0), (9, 400)]),
                                     (dict(group=3, kv_heads=3, dim=64, page=32), [(1, 5000), (100, 100), (5, 2), (2, 1)]),
                                     (dict(group=16, kv_heads=1, dim=256), [(1, 700), (9, 9), (2, 65)]),
                                     (dict(group=17, kv_heads=1), [(1, 300), (8, 90)])])
def test_prompts_among_single_tokens(gpu, kw, lens, call):
    """Long caches: the sequences of up to 16 rows x heads are the few-rows form's, the others the
    prompt form's, with and without pieces; and many such sequences, none of them in pieces."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, lens, **kw).fill(gpu)
    args = (c.cache, c.table, c.seq, c.cu)
    assert nv.mxfp4_attention_workspace_bytes(*args, c.tokens, c.heads, 1 << 13) > 0
    out = nv.mxfp4_attention(c.q, *args, max_kv=1 << 13, **call)
    c.check(out, **call)
    assert torch.equal(out, nv.mxfp4_attention(c.q, *args, max_kv=1 << 13, **call))
    c.check(nv.mxfp4_attention(c.q, *args, max_kv=1 << 17, **call), **call)
    own = torch.cat([c.q, torch.full_like(c.q[:2], 7.0)])  # its own output, with rows of no sequence
    nv.mxfp4_attention(own, *args, max_kv=1 << 17, out=own, **call)
    c.check(own[:c.tokens], **call)
    assert (own[c.tokens:] == 7.0).all()


@pytest.mark.parametrize("kv_heads,singles,prompt", [(2, 520, 3000), (8, 139, 600)])
def test_many_single_tokens_and_a_prompt(gpu, kv_heads, singles, prompt):
    """520: so many that the average makes it one launch of the few-rows form, the prompt with it.
    139 of 8 heads: the prompt form, and as many workgroups of the other as are wanted already."""
    import nvfp4_block_scaled_swiglu_amd as nv
    lens = [(1, 3 + i % 40) for i in range(singles)] + [(prompt, prompt)] + [(1, 20)] * 9
    c = Case(gpu, lens, group=4, dim=64, kv_heads=kv_heads).fill(gpu)
    c.check(nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu, max_kv=1 << 13))
