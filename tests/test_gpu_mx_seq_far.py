"""GPU: the operators around the cache where offsets pass 32 bits: pages behind 4 GiB of codes, rows behind
2^32 elements of the packed tensors."""
import numpy as np
import pytest

from tests import mx_ref, mx_seq_ref as ref, parity
from tests.test_gpu_mx_rope import check, rotation

pytestmark = pytest.mark.gpu

PAGES, PAGE, HEADS, DIM = 140000, 64, 8, 128  # 4.6e9 bytes of codes of keys


def test_pages(gpu):
    """Appended to a far page, copied to a near one and back, read by attention behind a prefix that lies there."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    cache = nv.empty_mxfp4_cache(PAGES, PAGE, HEADS, DIM, gpu)
    assert cache.k_codes.numel() > 1 << 32
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=gpu)  # noqa: E731
    far = PAGES - 1
    rng = np.random.default_rng(0)
    bits = [mx_ref.f64_to_bits(rng.standard_normal((70, HEADS, DIM))) for _ in range(3)]
    q, k, v = (parity.to_device_bf16(b, gpu) for b in bits)
    batch = (ints(far, far - 1)[None], ints(70), ints(0, 70))
    rot, freqs, _ = rotation(gpu, 128)
    rot.axes = None
    got = nv.mxfp4_norm_rope_append(cache, q, k, v, *batch, rot, eps=1e-6)
    angle = ref.turns(np.arange(70)[:, None], freqs)
    check(got, bits[0], angle, eps=1e-6)
    want = [mx_ref.round_trip(mx_ref.f64_to_bits(ref.norm_rope(mx_ref.bits_to_f64(bits[1]), angle, eps=1e-6)[0])),
            mx_ref.round_trip(bits[2])]

    def same(table):
        for t, w in zip(nv.mxfp4_cache_read(cache, table, ints(70), ints(0, 70), 70), want):
            np.testing.assert_array_equal(t.double().cpu().numpy(), w)

    same(batch[0])
    nv.mxfp4_cache_copy(cache, ints(far, far - 1, -1), ints(0, 1, 5))
    same(ints(0, 1)[None])
    nv.mxfp4_cache_copy(cache, ints(0, 1), ints(far - 2, far - 3))
    same(ints(far - 2, far - 3)[None])
    # two sequences behind the far page; their own tokens on a near one and a far one
    table = torch.stack([ints(-1, 1), ints(-1, far - 3)])
    x = got[-2:].contiguous()
    out = nv.mxfp4_attention_prefix(x, cache, table, ints(70, 70), ints(0, 1, 2), ints(far)[None], ints(64), ints(0, 2))
    o, tol = mx_ref.attention(x.double().cpu()[1:], *(torch.from_numpy(w) for w in want), DIM ** -0.5)
    assert bool(((out.double().cpu()[1:] - o).abs() <= tol).all())
    # pages given out at the far end
    pages = nv.empty_mxfp4_pages(2, 40, PAGES, PAGE, gpu)
    pages.refs.fill_(1)
    pages.refs[-30:] = 0
    done, _, _ = nv.mxfp4_pages_reserve(pages, ints(1, 0), ints(64 * 20, 64 * 10))
    assert done.tolist() == [1, 1] and pages.block_table[1, :20].tolist() == list(range(PAGES - 30, PAGES - 10))
    assert pages.block_table[0, :10].tolist() == list(range(PAGES - 10, PAGES))


def test_rows(gpu):
    """A row stride that puts the last row behind 2^32 elements, in and out."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    stride = 1 << 30
    rows = 5
    base = torch.empty((rows - 1) * stride + 2 * 64, dtype=torch.bfloat16, device=gpu)
    x = base.as_strided((rows, 2, 64), (stride, 64, 1))
    bits = mx_ref.f64_to_bits(np.random.default_rng(1).standard_normal((rows, 2, 64)))
    x.copy_(parity.to_device_bf16(bits, gpu))
    rot, freqs, which = rotation(gpu, 64)
    pos = np.arange(rows)[:, None]
    p = torch.arange(rows, dtype=torch.int32, device=gpu)
    check(nv.mxfp4_norm_rope(x, rot, p, eps=1e-6), bits, ref.turns(pos, freqs, which), eps=1e-6)
    assert nv.mxfp4_norm_rope(x, rot, p, eps=1e-6, out=x) is x
    check(x.contiguous(), bits, ref.turns(pos, freqs, which), eps=1e-6)
