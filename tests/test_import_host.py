"""Host-side checks of what the package needs to be imported, in processes of their own."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT_TORCH = "import sys; sys.modules['torch'] = None\n"

MXFP4_NAMES = """Mxfp4Cache Mxfp4Pages Mxfp4Rotation Mxfp4Tensor empty_mxfp4 empty_mxfp4_cache empty_mxfp4_pages mxfp4_attention
    mxfp4_attention_prefix mxfp4_attention_prefix_workspace_bytes mxfp4_attention_workspace_bytes mxfp4_cache_append mxfp4_cache_copy
    mxfp4_cache_read mxfp4_dequantize mxfp4_gemm_bf16out mxfp4_norm_rope mxfp4_norm_rope_append mxfp4_pages_compact
    mxfp4_pages_compact_workspace_bytes mxfp4_pages_fork mxfp4_pages_free mxfp4_pages_reserve mxfp4_pages_reserve_workspace_bytes
    mxfp4_qdata_bytes mxfp4_quantize mxfp4_quantize_swiglu mxfp4_rotation mxfp4_scale_bytes mxfp4_scale_cols""".split()


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


def test_without_torch():
    """The package, its build module, the library, sizes and records of the C functions."""
    out = run(WITHOUT_TORCH + """
import ctypes
import nvfp4_block_scaled_swiglu_amd as nv
import nvfp4_block_scaled_swiglu_amd.build
print(nv.nvfp4_padded_rows(129), nv.lib().mxfp4_scale_bytes(1, 32), nv.mxfp4_scale_bytes(129, 160), nv.mxfp4_qdata_bytes(3, 64),
      nv.mxfp4_scale_cols(32), nv.lib().mxfp4_pages_free(None, None, None, 1, None))
""")
    assert out == ["144", "512", "2048", "96", "4", "1"]


def test_operators_without_torch():
    """Named, and an ImportError that says what is missing."""
    out = run(WITHOUT_TORCH + """
import nvfp4_block_scaled_swiglu_amd as nv
print('mxfp4_attention' in dir(nv))
try:
    nv.mxfp4_attention
except ImportError as e:
    print(e.name)
""")
    assert out == ["True", "torch"]


def test_torch_is_not_loaded_by_the_import():
    assert run("import sys, nvfp4_block_scaled_swiglu_amd, nvfp4_block_scaled_swiglu_amd.build; print('torch' in sys.modules)") == ["False"]


def test_names():
    """All of them from the package, the modules among them, and what it has not is an AttributeError."""
    pytest.importorskip("torch")
    out = run(f"""
import nvfp4_block_scaled_swiglu_amd as nv
names = {MXFP4_NAMES!r}
assert set(names) <= set(dir(nv)) and set(names) <= set(nv.__all__)
for n in names:
    x = getattr(nv, n)
    assert x is getattr(nv, n) and x.__name__ == n, n
assert nv.mxfp4.mxfp4_attention is nv.mxfp4_attention and nv.mxfp4_pages.Mxfp4Pages is nv.Mxfp4Pages
assert nv.mxfp4_rope.mxfp4_rotation is nv.mxfp4_rotation
assert not hasattr(nv, 'mxfp4_nothing')
from nvfp4_block_scaled_swiglu_amd import *
assert mxfp4_cache_copy is nv.mxfp4_cache_copy and nvfp4_quantize is nv.nvfp4_quantize
print('fine')
""")
    assert out == ["fine"]


@pytest.mark.gpu
def test_library_before_torch(gpu):
    """The library loaded first, by a size; both then work on one HIP runtime."""
    out = run("""
import nvfp4_block_scaled_swiglu_amd as nv
nv.lib()
import torch
x = torch.ones(64, 64, device='cuda', dtype=torch.bfloat16)
print(bool((nv.mxfp4_dequantize(nv.mxfp4_quantize(x)) == 1).all()))
""")
    assert out == ["True"]
