"""GPU: what the MXFP4 binding refuses before the library is called."""
import pytest

from tests.test_gpu_mx_attention import Case

pytestmark = pytest.mark.gpu


def test_numbers_beyond_64_bits(gpu):
    """They would be cut to their low 64 bits: a window of 2^64 + 3 to one of 3."""
    import torch
    import nvfp4_block_scaled_swiglu_amd as nv
    c = Case(gpu, [(2, 20)], group=2).fill(gpu)
    args = (c.cache, c.table, c.seq, c.cu)
    for kw in (dict(window=2 ** 64 + 3), dict(window=3, sinks=2 ** 64), dict(max_kv=2 ** 63), dict(max_kv=2 ** 64 + 20),
               dict(window=-2 ** 64)):
        with pytest.raises(ValueError):
            nv.mxfp4_attention(c.q, *args, **kw)
        with pytest.raises(ValueError):
            nv.mxfp4_attention_workspace_bytes(*args, 2, c.heads, **{"max_kv": 20, **kw})
    with pytest.raises(ValueError):
        nv.mxfp4_attention_workspace_bytes(*args, 2 ** 64 + 2, c.heads, 20)
    t = nv.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16, device=gpu))
    for rows, k in ((4 - 2 ** 64, 64), (4, 64 - 2 ** 64)):
        with pytest.raises(ValueError):
            nv.mxfp4_dequantize(nv.Mxfp4Tensor(t.qdata, t.scales, rows, k))
    most = 2 ** 63 - 1
    c.check(nv.mxfp4_attention(c.q, *args, max_kv=most, window=most, sinks=most))
