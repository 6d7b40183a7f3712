"""The MXFP4 product in every form that its rules choose: the few-rows forms by rows and columns,
whole tiles, halves and quarters, alone and behind whole tiles. Sizes with odd edges and K of an
odd number of blocks, against float64."""
import pytest

from tests.test_gpu_mx_gemm import compare, operand

CUS = 256
SHAPES = [
    # few rows: 16-row tiles of A x 16-column tiles a workgroup
    (16, 777, 416), (5, 5130, 288), (16, 10250, 160), (1, 10241, 1056),
    (17, 333, 288), (20, 5130, 416), (32, 10250, 288), (20, 10243, 160),
    (33, 1001, 160), (50, 5130, 288), (64, 5121, 1056),
    # 33 to 64 rows of a wide weight: tiles
    (48, 10250, 288), (64, 16385, 160),
    # quarters, halves, whole tiles; each with one K pair, more pairs than stages, and in between
    (65, 129, 288), (700, 1500, 1056),
    (1021, 5301, 288), (300, 16400, 160), (1021, 5301, 1056),
    (1500, 7100, 288), (1500, 7100, 1056), (600, 15000, 32),
    (4096, 4096, 160), (4096, 4096, 544),
    # a whole round and halves, a whole round and quarters, and nearly two whole rounds
    (4700, 4400, 416), (4700, 4400, 1056), (4099, 4100, 416), (5121, 5121, 288),
]


def forms(m, n):
    """What a call of these sizes runs, by the rules at launch_mx_gemm and launch_tiles."""
    if m <= 32 or (m <= 64 and n < 10240):
        rows = 1 if m <= 16 else 2 if m <= 32 else 4
        return {("few", rows, 4 if n >= 10240 and rows < 4 else 2 if n >= 5120 else 1)}
    total = -(-m // 256) * -(-n // 256)
    last = total % CUS
    parts = 4 if last * 4 <= CUS else 2 if last * 2 <= CUS else 1
    whole = total if parts == 1 else total - last
    if whole == 0:
        return {("parts alone", parts)}
    return {("whole", 1)} | ({("behind whole", parts)} if whole < total else set())


def test_every_form_is_among_the_shapes():
    want = {("few", r, c) for r in (1, 2, 4) for c in (1, 2, 4)} - {("few", 4, 4)}
    want |= {("parts alone", 2), ("parts alone", 4), ("whole", 1), ("behind whole", 2), ("behind whole", 4)}
    assert set().union(*(forms(m, n) for m, n, _ in SHAPES)) == want
    # whole tiles alone, in a round that they fill and in one that they do not
    alone = [(-(-m // 256) * -(-n // 256)) % CUS for m, n, _ in SHAPES if forms(m, n) == {("whole", 1)}]
    assert 0 in alone and any(CUS // 2 < x for x in alone)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(gpu, m, n, k):
    """Into a tensor of its own, and into rows that are not 16-byte aligned, beside others."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    a, av = operand(m, k, m + n, gpu)
    w, wv = operand(n, k, m + n + 1, gpu, 0.02)
    out = nv.mxfp4_gemm_bf16out(a, w)
    compare(out, av, wv, k)
    hold = torch.full((m + 1, n + 5), 7.0, dtype=torch.bfloat16, device=gpu)
    nv.mxfp4_gemm_bf16out(a, w, out=hold[:m, 3:3 + n])
    assert torch.equal(hold[:m, 3:3 + n], out)  # the same sums
    hold[:m, 3:3 + n] = 7.0
    assert bool((hold == 7.0).all())
