"""GPU: lengths outside what a slot's row of the block table holds."""
import pytest

pytestmark = pytest.mark.gpu


def begun(gpu):
    """Slots of up to 48 tokens: 0 holds 48 but says 1,000, 1 holds 20, 2 is empty, 3 says -7."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    p = nv.empty_mxfp4_pages(4, 3, 20, 16, gpu)
    assert nv.mxfp4_pages_reserve(p, ints([0, 1]), ints([48, 20]))[0].tolist() == [1, 1]
    p.seq_lens[0] = 1000
    p.seq_lens[3] = -7
    return nv, p, ints


def lens(p):
    return p.seq_lens.clamp(0, 48).tolist()


@pytest.mark.parametrize("raw", [49, 1000, 2 ** 31 - 1])
def test_lengths_are_clamped(gpu, raw):
    """A length counts as max_pages * page_size at most, and as 0 at least, in every operator."""
    import torch
    nv, p, ints = begun(gpu)
    p.seq_lens[0] = raw
    table, refs = p.block_table.clone(), p.refs.clone()
    # not longer than 48: nothing to cut back
    nv.mxfp4_pages_free(p, ints([0]), ints([48]))
    assert lens(p) == [48, 20, 0, 0] and int(p.seq_lens[0]) == raw
    assert torch.equal(p.block_table, table) and torch.equal(p.refs, refs)
    # of 48 tokens: may stay as it is, cannot become shorter or longer
    done, src, dst = nv.mxfp4_pages_reserve(p, ints([0, 1]), ints([48, 20]))
    assert done.tolist() == [1, 1] and src.tolist() == [-1, -1] == dst.tolist()
    assert nv.mxfp4_pages_reserve(p, ints([0, 3]), ints([47, -1]))[0].tolist() == [0, 0]
    assert nv.mxfp4_pages_reserve(p, ints([0, 3]), ints([49, 0]))[0].tolist() == [0, 1]
    assert lens(p) == [48, 20, 0, 0]
    assert torch.equal(p.block_table, table) and torch.equal(p.refs, refs)
    # a child has as many tokens as its parent, and none of one that says less than none
    assert nv.mxfp4_pages_fork(p, ints([0]), ints([2])).tolist() == [1]
    assert p.seq_lens[2].item() == 48 and torch.equal(p.block_table[2], table[0])
    assert p.refs.tolist() == [2, 2, 2, 1, 1] + [0] * 15
    # cut back to less than 48
    nv.mxfp4_pages_free(p, ints([0]), ints([20]))
    assert lens(p) == [20, 20, 48, 0] and p.refs.tolist() == [2, 2, 1, 1, 1] + [0] * 15
    assert p.block_table[0].tolist() == [0, 1, -1]


def test_a_number_kept_beyond_the_row(gpu):
    """More than a row holds, and less than what the length says: not longer, so nothing is cut."""
    nv, p, ints = begun(gpu)
    nv.mxfp4_pages_free(p, ints([0, 1, 0]), ints([60, 60, 500]))
    assert p.seq_lens.tolist() == [1000, 20, 0, -7] and p.refs.tolist() == [1] * 5 + [0] * 15


def test_a_child_of_a_slot_without_tokens(gpu):
    nv, p, ints = begun(gpu)
    assert nv.mxfp4_pages_fork(p, ints([3]), ints([2])).tolist() == [1]
    assert p.seq_lens.tolist() == [1000, 20, 0, -7]


def test_lengths_are_clamped_in_long_lists(gpu):
    """Of more than 128 entries, which a launch of its own enters."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    n = 200
    p = nv.empty_mxfp4_pages(n, 3, 3 * n, 16, gpu)
    every = torch.arange(n, dtype=torch.int32, device=gpu)
    assert bool((nv.mxfp4_pages_reserve(p, every, torch.full_like(every, 48))[0] == 1).all())
    p.seq_lens[::2] = 1000
    p.seq_lens[1::4] = 33
    want = torch.where(every % 4 == 1, 47, 48).to(torch.int32)
    done, src, dst = nv.mxfp4_pages_reserve(p, every, want)
    assert bool((done == 1).all()) and bool((src == -1).all()) and bool((dst == -1).all())
    assert torch.equal(p.seq_lens.clamp(0, 48), want) and bool((p.refs == 1).all())
    assert nv.mxfp4_pages_reserve(p, every, torch.full_like(every, 47))[0].tolist() == (every % 4 == 1).int().tolist()


@pytest.mark.parametrize("size", [2 ** 64 + 16, 2 ** 63, -2 ** 64 + 16, -2 ** 63 - 1])
def test_page_size_beyond_64_bits(gpu, size):
    """Refused, not cut to 64 bits on its way into the library."""
    nv, p, ints = begun(gpu)
    p.page_size = size
    before = [t.clone() for t in (p.block_table, p.seq_lens, p.refs)]
    for call in (lambda: nv.mxfp4_pages_free(p, ints([0])), lambda: nv.mxfp4_pages_fork(p, ints([0]), ints([2])),
                 lambda: nv.mxfp4_pages_reserve(p, ints([0]), ints([48])), lambda: nv.mxfp4_pages_compact(p),
                 lambda: nv.mxfp4_pages_reserve_workspace_bytes(p, 1), lambda: nv.mxfp4_pages_compact_workspace_bytes(p)):
        with pytest.raises(ValueError):
            call()
    assert all(bool((a == b).all()) for a, b in zip(before, (p.block_table, p.seq_lens, p.refs)))
