"""GPU: the pages' bookkeeping against lists, and copies of pages, byte for byte."""
import numpy as np
import pytest

from tests import mx_seq_ref as ref

pytestmark = pytest.mark.gpu


def ints(gpu, x):
    import torch
    return torch.tensor(np.asarray(x, dtype=np.int64).reshape(-1), dtype=torch.int32, device=gpu)


def same(pages, model):
    np.testing.assert_array_equal(pages.seq_lens.cpu().numpy(), model.lens)
    np.testing.assert_array_equal(pages.block_table.cpu().numpy(), model.table)
    np.testing.assert_array_equal(pages.refs.cpu().numpy(), model.refs)


class Both:
    """The library's record and the lists, after the same steps."""

    def __init__(self, gpu, slots, max_pages, num_pages, page):
        import nvfp4_block_scaled_swiglu_amd as nv
        self.gpu, self.nv = gpu, nv
        self.pages = nv.empty_mxfp4_pages(slots, max_pages, num_pages, page, gpu)
        self.model = ref.Pages(slots, max_pages, num_pages, page)

    def check(self):
        same(self.pages, self.model)

    def reserve(self, slots, lens):
        got = self.nv.mxfp4_pages_reserve(self.pages, ints(self.gpu, slots), ints(self.gpu, lens))
        want = self.model.reserve(list(slots), list(lens))
        for g, w in zip(got, want):
            assert g.tolist() == [int(x) for x in w]
        self.check()
        return got

    def fork(self, parents, children):
        got = self.nv.mxfp4_pages_fork(self.pages, ints(self.gpu, parents), ints(self.gpu, children))
        assert got.tolist() == self.model.fork(list(parents), list(children))
        self.check()

    def free(self, slots, keep=None):
        self.nv.mxfp4_pages_free(self.pages, ints(self.gpu, slots), None if keep is None else ints(self.gpu, keep))
        self.model.free(list(slots), keep)
        self.check()

    def compact(self, in_place):
        before = [t.clone() for t in (self.pages.block_table, self.pages.refs)]
        after, src, dst, used = self.nv.mxfp4_pages_compact(self.pages, out=self.pages if in_place else None)
        if not in_place:  # the old record stays
            assert all(bool((a == b).all()) for a, b in zip(before, (self.pages.block_table, self.pages.refs)))
        want = self.model.compact()
        assert src.tolist() == want[0] and dst.tolist() == want[1] and used.tolist() == [want[2]]
        self.pages = after
        self.check()


def test_each_step(gpu):
    b = Both(gpu, 8, 6, 40, 16)
    b.reserve([3, 0, 5], [50, 16, 0])            # 4 pages, 1, none
    b.reserve([3, 0, 0, 3], [50, 17, 40, 60])    # nothing; one; listed twice; listed twice
    b.fork([3, 3, 0], [1, 2, 4])                 # a shared last page, and one not full
    b.reserve([1, 3, 4], [51, 64, 32])           # copies of it; 4's fits, and copies too
    b.reserve([2], [52])                         # the last one that holds it: no copy
    b.free([1, 1, 9, -1], [33, 20, 0, 0])        # cut back twice; no such slots
    b.free([3, 4, 2], [64, 100, -5])             # not longer; not longer; to nothing
    b.reserve([6], [6 * 16])
    b.reserve([6], [6 * 16 + 1])                 # more than a row holds
    b.reserve([6, 3], [5, 63])                   # shorter than it is
    b.compact(False)
    b.compact(True)                              # nothing left to move


def test_pairs_that_are_not_forked(gpu):
    b = Both(gpu, 9, 4, 40, 16)
    b.reserve([0, 1], [40, 20])
    b.fork([0, 1, 0, 1, 0, -1, 1, 9], [2, 2, 1, 3, 0, 4, -1, 5])  # 2 twice, 1 is a parent and holds pages, 0 its own, none
    b.fork([7, 0], [8, 7])                                       # 7 is a child: not a parent in the same call
    b.fork([4], [5])                                             # of an empty sequence: an empty one
    b.fork([0] * 3, [3, 4, 6])


def test_too_few_pages(gpu):
    """Entries are served in order while what they need up to there was free; one that needs
    nothing always is."""
    b = Both(gpu, 8, 10, 13, 16)
    b.reserve([0, 1, 2, 3, 4], [80, 96, 48, 16, 16])   # 5, 6, then 3 of the 2 left, and all behind them
    b.reserve([0, 2, 3], [80, 0, 32])
    b.fork([0], [5])
    b.free([1])
    b.reserve([5, 0, 1, 2], [81, 81, 300, 1])
    b.reserve([2, 3], [160, 160])
    b.compact(True)


@pytest.mark.parametrize("seed,slots,most,num,page", [(0, 20, 12, 100, 16), (1, 64, 30, 700, 64), (2, 5, 3, 9, 128), (3, 40, 70, 1500, 16), (4, 12, 700, 5000, 16), (5, 300, 9, 1800, 32)])
def test_random_steps(gpu, seed, slots, most, num, page):
    rng = np.random.default_rng(seed)
    b = Both(gpu, slots, most, num, page)
    for _ in range(25):
        n = int(rng.integers(1, slots + 1))
        some = rng.permutation(slots)[:n]
        kind = rng.integers(0, 6)
        if kind <= 1:
            b.reserve(some, [min(int(b.model.lens[s]) + int(rng.integers(0, 3 * page)), most * page + 1) for s in some])
        elif kind <= 3:
            b.fork(rng.permutation(slots)[:n], some)
        elif kind == 4:
            some = some[:max(1, n // 3)]
            b.free(some, None if rng.random() < 0.5 else [int(rng.integers(0, most * page)) for _ in some])
        else:
            b.compact(bool(rng.integers(2)))


@pytest.mark.parametrize("n,num", [(1023, 5000), (1025, 9000), (3000, 400000), (3000, 262145)])
def test_many(gpu, n, num):
    """Lists longer than the planning workgroup, and more pages than its bitmap holds."""
    import torch
    b = Both(gpu, n, 4, num, 16)
    held = np.random.default_rng(n).random(num) < 0.97  # by others, below; the last pages are free
    held[-2 * n:] = False
    b.pages.refs.copy_(torch.from_numpy(held.astype(np.int32)))
    b.model.refs[:] = held
    rng = np.random.default_rng(0)
    order = rng.permutation(n)
    lens = rng.integers(0, 40, n)
    slow = b.model.reserve
    got = b.nv.mxfp4_pages_reserve(b.pages, ints(gpu, order), ints(gpu, lens))
    done = lens >= 0
    free = np.flatnonzero(~held)
    need = -(-lens // 16)
    start = np.cumsum(need) - need
    assert need.sum() <= len(free) and slow is not None
    for i, s in enumerate(order):
        b.model.table[s, :need[i]] = free[start[i]:start[i] + need[i]]
        b.model.refs[free[start[i]:start[i] + need[i]]] = 1
        b.model.lens[s] = lens[i]
    assert got[0].tolist() == done.astype(int).tolist() and got[1].max().item() == -1 == got[2].max().item()
    b.check()
    b.compact(False)


def test_strided_rows(gpu):
    """A block table inside a wider one."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    wide = torch.full((4, 9), 77, dtype=torch.int32, device=gpu)
    wide[:, 2:7] = -1
    p = nv.Mxfp4Pages(wide[:, 2:7], torch.zeros(4, dtype=torch.int32, device=gpu), torch.zeros(30, dtype=torch.int32, device=gpu), 16)
    m = ref.Pages(4, 5, 30, 16)
    nv.mxfp4_pages_reserve(p, ints(gpu, [2, 0]), ints(gpu, [70, 33]))
    m.reserve([2, 0], [70, 33])
    nv.mxfp4_pages_fork(p, ints(gpu, [2]), ints(gpu, [3]))
    m.fork([2], [3])
    nv.mxfp4_pages_free(p, ints(gpu, [0]))
    m.free([0])
    after = nv.mxfp4_pages_compact(p)[0]
    same(p, m)
    m.compact()
    same(after, m)
    assert bool((wide[:, :2] == 77).all()) and bool((wide[:, 7:] == 77).all())


def test_compact_into_a_record(gpu):
    """Of the caller's, with lengths of its own and wider rows; one of another size is refused."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    b = Both(gpu, 3, 4, 20, 16)
    b.reserve([0, 1, 2], [60, 33, 20])
    b.free([0])
    wide = torch.full((3, 8), 77, dtype=torch.int32, device=gpu)
    out = nv.Mxfp4Pages(wide[:, 1:5], torch.full((3,), 9, dtype=torch.int32, device=gpu), torch.full((20,), 5, dtype=torch.int32, device=gpu), 16)
    assert nv.mxfp4_pages_compact(b.pages, out=out)[0] is out
    b.check()
    b.model.compact()
    same(out, b.model)
    assert bool((wide[:, :1] == 77).all()) and bool((wide[:, 5:] == 77).all())
    with pytest.raises(ValueError):
        nv.mxfp4_pages_compact(b.pages, out=nv.empty_mxfp4_pages(3, 4, 21, 16, gpu))


def cache_of(gpu, pages, page, heads, dim, seed):
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = nv.empty_mxfp4_cache(pages, page, heads, dim, gpu)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in tensors(c):
        t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8, device=gpu, generator=g))
    return c


def tensors(c):
    return (c.k_codes, c.k_scales, c.v_codes, c.v_scales)


@pytest.mark.parametrize("pages,page,heads,dim", [(9, 16, 1, 64), (40, 64, 8, 128), (21, 32, 3, 256), (300, 16, 5, 128), (5, 4096, 2, 64)])
def test_copy(gpu, pages, page, heads, dim):
    """Within a cache and into another one, numbers out of range passed over."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    rng = np.random.default_rng(pages)
    order = rng.permutation(pages)
    half = pages // 2
    src, dst = order[:half].copy(), order[half:2 * half].copy()
    dead = rng.random(half) < 0.4
    src[dead] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31], int(dead.sum()))
    c = cache_of(gpu, pages, page, heads, dim, 1)
    want = [t.clone() for t in tensors(c)]
    for w in want:
        for a, b in zip(src, dst):
            if 0 <= a < pages:
                w[b] = w[a]
    assert nv.mxfp4_cache_copy(c, ints(gpu, src), ints(gpu, dst)) is c
    for t, w in zip(tensors(c), want):
        assert torch.equal(t, w)
    to = cache_of(gpu, pages + 7, page, heads, dim, 2)
    want = [t.clone() for t in tensors(to)]
    dst = np.where(rng.random(half) < 0.2, pages + 7, dst + 7)
    for w, f in zip(want, tensors(c)):
        for a, b in zip(src, dst):
            if 0 <= a < pages and b < pages + 7:
                w[b] = f[a]
    nv.mxfp4_cache_copy(c, ints(gpu, src), ints(gpu, dst), target=to)
    for t, w in zip(tensors(to), want):
        assert torch.equal(t, w)


def test_copy_of_a_few_among_many(gpu):
    """A list whose pairs lie far apart, longer than one look of every workgroup."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = cache_of(gpu, 64, 16, 2, 64, 3)
    want = [t.clone() for t in tensors(c)]
    n = 400001
    src, dst = torch.full((2, n), -1, dtype=torch.int32, device=gpu)
    for i, at in enumerate((0, 1, 63, 2047, 131072, 262143, n - 1)):
        src[at], dst[at] = i, 63 - i
        for w in want:
            w[63 - i] = w[i]
    nv.mxfp4_cache_copy(c, src, dst)
    for t, w in zip(tensors(c), want):
        assert torch.equal(t, w)
