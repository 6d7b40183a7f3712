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
