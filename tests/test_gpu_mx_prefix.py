"""GPU: attention behind shared prefixes, against float64 row by row."""
import numpy as np
import pytest

from tests import mx_ref, parity
from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


class Shared(Case):
    """A batch whose last sequences, without rows, are the prefixes. lens: of the others; prefixes: their
    tokens; groups: where each one's group starts, and the end. Own pages below the shared tokens hold
    other tokens than the prefix, or are not there (torn)."""

    def __init__(self, gpu, lens, prefixes, starts, torn=False, **kw):
        import torch
        super().__init__(gpu, lens + [(0, n) for n in prefixes], **kw)
        self.fill(gpu)
        self.count, self.prefixes, self.starts = len(lens), prefixes, starts
        self.prefix_table = self.table[self.count:].clone()
        self.prefix_lens = torch.tensor(prefixes, dtype=torch.int32, device=gpu)
        self.group_starts = torch.tensor(starts, dtype=torch.int32, device=gpu)
        if torn:
            for i in range(self.count):
                self.table[i, :self.shared(i)[1] // self.page] = -1

    def shared(self, i, causal=True):
        """(group, tokens that sequence i reads through its table)"""
        q, kv = self.lens[i]
        for g, n in enumerate(self.prefixes):
            if self.starts[g] <= i < self.starts[g + 1]:
                s = n // 64 * 64
                return g, s if s <= (kv - q + 1 if causal else kv) else 0
        return -1, 0

    def run(self, **kw):
        import nvfp4_block_scaled_swiglu_amd as nv
        return nv.mxfp4_attention_prefix(self.q, self.cache, self.table, self.seq, self.cu, self.prefix_table, self.prefix_lens,
                                         self.group_starts, **kw)

    def check_shared(self, out, causal=True, scale=None, hidden=None):
        import torch
        k, v = (torch.from_numpy(mx_ref.round_trip(b)) for b in (self.k_bits, self.v_bits))
        q = torch.from_numpy(mx_ref.bits_to_f64(self.q_bits))
        got = out.double().cpu()
        base = np.concatenate([[0], np.cumsum([kv for _, kv in self.lens])])
        at = 0
        for i, (n, kv) in enumerate(self.lens[:self.count]):
            g, s = self.shared(i, causal)
            p = base[self.count + g] if s else 0
            kk, vv = (torch.cat([x[p:p + s], x[base[i] + s:base[i] + kv]]) for x in (k, v))
            h = None
            if hidden is not None:
                h = torch.zeros(kv, dtype=torch.bool)
                h[:s] = hidden[self.count + g][:s] if s else False
            want, tol = mx_ref.attention(q[at:at + n], kk, vv, self.dim ** -0.5 if scale is None else scale, causal=causal, hidden=h)
            x = got[at:at + n]
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(x), nan), i
            off = torch.where(nan, 0.0, (x - want).abs())
            assert bool((off <= torch.where(nan, 1.0, tol)).all()), (i, float((off / tol.clamp(min=1e-300)).max()))
            at += n


SHAPES = [
    # single tokens, one group: few packed rows, then many
    (dict(dim=128, page=16, group=1), [(1, 90 + i) for i in range(5)], [70], [0, 5]),
    (dict(dim=128, page=64, group=7, kv_heads=2), [(1, 300 + 9 * i) for i in range(12)], [290], [0, 12]),
    (dict(dim=64, page=32, group=4, kv_heads=2), [(1, 200 + i) for i in range(7)], [200], [0, 7]),
    (dict(dim=256, page=16, group=3, kv_heads=1), [(1, 140 + i) for i in range(3)], [128], [0, 3]),
    (dict(dim=256, page=128, group=4, kv_heads=1), [(2, 500 + 30 * i) for i in range(6)], [449], [0, 6]),
    # a prefix that ends inside a page, one of less than 64 tokens, one of none
    (dict(dim=128, page=128, group=2), [(1, 400), (2, 330), (1, 80), (1, 70), (1, 9)], [330, 63, 0], [0, 2, 4, 5]),
    # sequences before, between (a group without any) and behind the groups; rows that share nothing
    (dict(dim=64, page=16, group=5), [(1, 30), (1, 100), (3, 120), (1, 64), (1, 1), (2, 77)], [64, 64, 128], [1, 3, 3, 4]),
    # drafts and questions: rows that see part of their own tokens
    (dict(dim=128, page=32, group=3, kv_heads=2), [(5, 205), (9, 209), (30, 240), (1, 193)], [199], [0, 4]),
    (dict(dim=64, page=64, group=2, kv_heads=2), [(150, 300), (40, 300), (129, 257)], [130], [0, 3]),
    # just everything shared but the row's own token; one token more; one less
    (dict(dim=128, page=64, group=1), [(1, 128), (1, 129), (1, 127), (2, 129), (2, 128)], [128], [0, 5]),
]


@pytest.mark.parametrize("torn", [False, True])
@pytest.mark.parametrize("kw,lens,prefixes,starts", SHAPES)
def test_against_the_definition(gpu, kw, lens, prefixes, starts, torn):
    c = Shared(gpu, lens, prefixes, starts, torn, **kw)
    c.check_shared(c.run())
    c.check_shared(c.run(max_prefix=100000, max_own=100000))  # in many pieces, of which some are empty
    c.check_shared(c.run(max_prefix=1, max_own=1))
    if not torn:
        c.check_shared(c.run(causal=False), causal=False)
    c.check_shared(c.run(scale=2.0), scale=2.0)


def test_padded_batch(gpu):
    """Slots without a sequence (length 0, a row each), a sequence shorter than its rows, rows of no
    sequence: zeros, and what out held."""
    import torch
    c = Shared(gpu, [(1, 0), (1, 200), (1, 0), (3, 2), (1, 150)], [130], [0, 5], dim=128, page=16, group=2)
    q = torch.cat([c.q, c.q[:4]])
    out = torch.full_like(q, 9.0)
    import nvfp4_block_scaled_swiglu_amd as nv
    got = nv.mxfp4_attention_prefix(q, c.cache, c.table, c.seq, c.cu, c.prefix_table, c.prefix_lens, c.group_starts, out=out)
    assert got is out and bool((out[7:] == 9).all())
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all()) and bool((out[3] == 0).all())
    c.check_shared(out[:7])


def test_pages_that_are_not_there(gpu):
    """Of a prefix: nobody sees them, and garbage on them reaches nobody; of all of it; and NaN blocks
    in a prefix reach everybody behind it."""
    import torch
    c = Shared(gpu, [(1, 300), (2, 280), (1, 270)], [256], [0, 3], dim=128, page=32, group=2)
    c.prefix_table[0, 2] = -1
    c.prefix_table[0, 5] = c.cache.num_pages
    hidden = [torch.zeros(kv, dtype=torch.bool) for _, kv in c.lens]
    hidden[3][64:96] = True
    hidden[3][160:192] = True
    c.check_shared(c.run(), hidden=hidden)
    c.prefix_table.fill_(-1)
    hidden[3][:] = True
    c.check_shared(c.run(), hidden=hidden)
    c = Shared(gpu, [(1, 300), (2, 280)], [256], [0, 1], dim=64, page=32, group=2)
    c.cache.v_scales[c.prefix_table[0, 1].item(), 1, 7] = 255  # of head 1's values: one token
    out = c.run()
    assert bool(torch.isnan(out[0, 2:]).all()) and not bool(torch.isnan(out[0, :2]).any()) and not bool(torch.isnan(out[1:]).any())


def test_no_groups(gpu):
    """Equal to mxfp4_attention, bit for bit."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Shared(gpu, [(1, 300), (40, 280)], [64], [0, 1], dim=128, page=32, group=2)
    got = nv.mxfp4_attention_prefix(c.q, c.cache, c.table, c.seq, c.cu, c.prefix_table[:0], c.prefix_lens[:0], c.group_starts[:1])
    assert torch.equal(got, nv.mxfp4_attention(c.q, c.cache, c.table, c.seq, c.cu))


@pytest.mark.parametrize("count,groups,q", [(63, 1, 1), (64, 1, 1), (70, 3, 2), (63, 63, 1), (64, 62, 3), (66, 64, 1), (130, 65, 1)])
def test_counts_around_a_wave(gpu, count, groups, q):
    """Sequences and groups are looked up 64 at a time, up to 63 of both at once."""
    starts = [g * count // groups for g in range(groups)] + [count - (groups == 62)]  # (of 62 the last sequence is in none)
    lens = [(1 + i % q, 130 + i % 9 + 64 * (i % 3)) for i in range(count)]
    c = Shared(gpu, lens, [128 - 64 * (g % 2) for g in range(groups)], starts, torn=True, dim=64, page=32, group=2)
    c.check_shared(c.run())


@pytest.mark.parametrize("before,behind", [(40000, 0), (0, 40000), (300, 300)])
def test_many_groups_without_sequences(gpu, before, behind):
    import torch
    c = Shared(gpu, [(1, 3000 + i) for i in range(3)], [2900], [0, 3], dim=128, page=64, group=4, kv_heads=2)
    c.prefix_table = torch.nn.functional.pad(c.prefix_table, (0, 0, before, behind), value=-1)
    c.prefix_lens = torch.nn.functional.pad(c.prefix_lens, (before, behind), value=64)
    c.group_starts = torch.nn.functional.pad(torch.nn.functional.pad(c.group_starts, (before, 0)), (0, behind), value=3)
    c.check_shared(c.run())


@pytest.mark.parametrize("dim,heads,per,q,prefix,own", [(128, 28, 24, 1, 20000, 900), (64, 16, 9, 3, 7001, 300), (128, 16, 6, 200, 2500, 400),
                                                        (256, 8, 16, 1, 3001, 200)])
def test_long(gpu, dim, heads, per, q, prefix, own):
    """Long prefixes in many pieces, against float64 on the card, by the tolerance of mx_ref.attention."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    kv_heads, page = 4, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    shared = -(-prefix // page)
    each = -(-(prefix % page + own) // page) + 1
    count = shared + per * each
    cache = nv.empty_mxfp4_cache(count, page, kv_heads, dim, gpu)
    full = prefix // page
    order = torch.randperm(count, generator=g, device=gpu).to(torch.int32)
    table = torch.full((per, full + each), -1, dtype=torch.int32, device=gpu)
    table[:, full:] = order[shared:].view(per, each)
    prefix_table = order[:shared][None].contiguous()
    lens = [full * page + own - 3 * i for i in range(per)]
    seq = torch.tensor(lens, dtype=torch.int32, device=gpu)
    cu = torch.arange(0, per * q + 1, q, dtype=torch.int32, device=gpu)
    everything = torch.arange(count, dtype=torch.int32, device=gpu)[:, None].contiguous()
    k, v = (torch.randn(count * page, kv_heads, dim, generator=g, device=gpu).bfloat16() for _ in range(2))
    starts = torch.arange(0, count * page + 1, page, dtype=torch.int32, device=gpu)
    whole = torch.full((count,), page, dtype=torch.int32, device=gpu)
    nv.mxfp4_cache_append(cache, k, v, everything, whole, starts)
    k, v = (x.double().view(count, page, kv_heads, dim) for x in nv.mxfp4_cache_read(cache, everything, whole, starts, count * page))
    x = torch.randn(per * q, heads, dim, generator=g, device=gpu).bfloat16()
    out = nv.mxfp4_attention_prefix(x, cache, table, seq, cu, prefix_table, torch.tensor([full * page], dtype=torch.int32, device=gpu),
                                    torch.tensor([0, per], dtype=torch.int32, device=gpu), max_own=own).double()
    group = heads // kv_heads
    for i in range(per):
        pages = torch.cat([prefix_table[0, :full], table[i, full:]]).long()
        kk, vv = (y[pages].flatten(0, 1)[:lens[i]] for y in (k, v))
        hidden = torch.arange(lens[i], device=gpu)[None] > torch.arange(lens[i] - q, lens[i], device=gpu)[:, None]
        for h in range(heads):
            y = x[i * q:(i + 1) * q, h].double()
            s = (y @ kk[:, h // group].t() * dim ** -0.5).masked_fill(hidden, -float("inf"))
            w = torch.softmax(s, -1)
            want = w @ vv[:, h // group]
            mag = (y.abs() @ kk[:, h // group].abs().t() * dim ** -0.5).amax(-1, keepdim=True)
            err = 2.0 ** -8 + 2.0 ** -14 + 2 * (dim + 2) * 2.0 ** -23 * mag
            tol = err * (w @ vv[:, h // group].abs()) + 2 * 2.0 ** -8 * want.abs() + 2.0 ** -100
            assert bool(((out[i * q:(i + 1) * q, h] - want).abs() <= tol).all()), (i, h)
