"""Host-side checks of the MXFP4 operators' limits: calls just inside them pass the validation
(without a GPU: report that there is no device), calls outside are refused with their status."""
import pytest

import nvfp4_block_scaled_swiglu_amd as nv
from tests.test_mx_host import ATTN, structs

NO_DEVICE = 5


@pytest.fixture
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible: a call that passes would run")


def attention(kw):
    c, b = structs(kw)
    return nv.lib().mxfp4_attention(c, b, *{**ATTN, **{n: v for n, v in kw.items() if n in ATTN}}.values())


def test_largest_scale(no_gpu):
    assert attention(dict(scale=2.0 ** 127)) == NO_DEVICE
    assert attention(dict(scale=1.5 * 2.0 ** 127)) == 1
    assert attention(dict(scale=2.0 ** -149)) == NO_DEVICE


@pytest.mark.parametrize("kw,status", [
    # what the sizes of a launch allow: (tokens * heads / kv_heads / 16 + batch) * kv_heads below 2^24
    (dict(b_tokens=262144, b_batch=1, c_heads=8, heads=64), NO_DEVICE),
    (dict(b_tokens=262144, b_batch=262144, c_heads=8, heads=64), NO_DEVICE),
    (dict(b_tokens=1 << 24, b_batch=1, c_heads=1, heads=8), NO_DEVICE),
    (dict(b_tokens=(1 << 24) - 17, b_batch=1, c_heads=1, heads=16), NO_DEVICE),
    (dict(b_tokens=(1 << 24) - 1, b_batch=1, c_heads=1, heads=16), 2),
    (dict(b_tokens=1, b_batch=1 << 21, c_heads=8, heads=8), 2),
    (dict(b_tokens=1 << 24, b_batch=1, c_heads=1, heads=128), 2),  # rows x heads of a group: 2^31
])
def test_rows_and_heads_of_an_attention(no_gpu, kw, status):
    wide = dict(qt=1 << 20, ot=1 << 20)
    assert attention({**wide, **kw}) == status
    c, b = structs(kw)
    size = nv.lib().mxfp4_attention_workspace_bytes(c, b, kw["heads"], 32, 0, 0)
    assert size == (0 if status == NO_DEVICE else -1)



@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_of_a_cache_call(no_gpu, dim):
    """A launch takes 2^24 - 1 workgroups of 2048 / head_dim rows."""
    most = ((1 << 24) - 1) * (2048 // dim)
    for tokens, status in ((most, NO_DEVICE), (most + 1, 2), ((1 << 31) - 1, 2)):
        c, b = structs(dict(c_dim=dim, b_tokens=tokens))
        for f in (nv.lib().mxfp4_cache_append, nv.lib().mxfp4_cache_read):
            assert f(c, b, 0x10000, 2 * dim, dim, 0x10000, 2 * dim, dim, None) == status


@pytest.mark.parametrize("group,some", [(16, True), (17, False), (40, False)])
def test_workspace_of_short_sequences(group, some):
    """Prompts that need no pieces, long caches: room for sequences of up to 16 rows x heads, which
    a group of more heads cannot have."""
    c, b = structs(dict(b_tokens=4000))
    size = nv.lib().mxfp4_attention_workspace_bytes(c, b, 2 * group, 1 << 14, 0, 0)
    assert (size > 0) == some


def test_strides_of_a_single_token(no_gpu):
    """One token of a heads-first tensor: its stride between tokens means nothing, and must not be
    made up beyond what is taken (2^31)."""
    import torch
    from nvfp4_block_scaled_swiglu_amd import mxfp4
    x = torch.empty((64, 1 << 20, 64), dtype=torch.bfloat16, device="meta").transpose(0, 1)
    for t in (x[5:6], x[5:6, :1], x[5:9]):
        tokens, heads, dim = t.shape
        strides = mxfp4._strides(t)
        assert strides[0] == t.stride(0) or tokens == 1
        assert strides[1] == t.stride(1) or heads == 1
        c, b = structs(dict(c_heads=heads, b_tokens=tokens))
        assert nv.lib().mxfp4_cache_read(c, b, 0x10000, *strides, 0x10000, *strides, None) == NO_DEVICE


@pytest.mark.parametrize("rows,k,status", [
    (((1 << 21) - 1) * 128, 512, NO_DEVICE), (((1 << 21) - 1) * 128 + 1, 512, 2), (((1 << 21) - 1) * 128, 544, 2),
    (128, 1 << 23, NO_DEVICE), (127 * 128, 1 << 23, NO_DEVICE), (129 * 128, 1 << 23, 2),
])
def test_size_of_a_matrix(no_gpu, rows, k, status):
    l, p = nv.lib(), 0x10000
    assert l.mxfp4_quantize(p, k, rows, k, p, p, None) == status
    assert l.mxfp4_quantize_swiglu(p, k, p, k, rows, k, p, p, None) == status
    assert l.mxfp4_dequantize(p, p, rows, k, p, k, None) == status
    assert l.mxfp4_gemm_bf16out(p, p, p, p, p, 64, rows, 64, k, None) == status
    assert l.mxfp4_gemm_bf16out(p, p, p, p, p, rows, 64, rows, k, None) == status


def test_size_of_a_product(no_gpu):
    f, p = nv.lib().mxfp4_gemm_bf16out, 0x10000
    assert f(p, p, p, p, p, 1 << 40, 64 << 12, 64 * 4095, 32, None) == NO_DEVICE
    assert f(p, p, p, p, p, 1 << 40, 64 << 12, 64 * 4096, 32, None) == 2
    assert f(p, p, p, p, p, (1 << 40) + 1, 64, 64, 32, None) == 2
