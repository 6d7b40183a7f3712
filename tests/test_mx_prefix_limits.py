"""Host-side check of the rows that a call of attention behind prefixes takes: its join has a workgroup of 256
threads for four rows x heads, and a launch 2^24 - 1 of them."""
import pytest

import nvfp4_block_scaled_swiglu_amd as nv
from tests.test_mx_host import structs
from tests.test_mx_seq_host import passed, prefix

MOST = 4 * ((1 << 24) - 1)


@pytest.mark.parametrize("tokens,status", [(MOST - 1, 0), (MOST, 0), (MOST + 1, 2), (MOST + 2, 2), (MOST + 3, 2), (MOST + 4, 2)])
@pytest.mark.parametrize("batch,groups", [(1, 1), (8388000, 1), (1, 8388000), (1, 0)])
def test_one_head(tokens, status, batch, groups):
    kw = dict(b_tokens=tokens, b_batch=batch, c_heads=1, heads=1, x_groups=groups)
    rc, size = prefix(kw)
    assert rc == passed(status)
    assert (size == -1) == (status != 0)


@pytest.mark.parametrize("heads,tokens,status", [(3, MOST // 3, 0), (3, MOST // 3 + 1, 2), (17, MOST // 17 - 1000000, 0), (17, MOST // 17 + 1, 2)])
def test_several_heads(heads, tokens, status):
    """MOST is 3 * 22369620: up to it with three heads."""
    kw = dict(b_tokens=tokens, b_batch=1, c_heads=heads, heads=heads, x_groups=1, ot=64 * heads, qt=64 * heads)
    rc, size = prefix(kw)
    assert rc == passed(status)
    assert (size == -1) == (status != 0)


def test_whole_calls_keep_theirs():
    """mxfp4_attention joins only where there are few rows."""
    c, b = structs(dict(b_tokens=MOST + 3, b_batch=1, c_heads=1))
    assert nv.lib().mxfp4_attention_workspace_bytes(c, b, 1, 1 << 17, 0, 0) == 0
