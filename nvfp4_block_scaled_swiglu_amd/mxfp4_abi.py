"""The C side of the MXFP4 operators (``include/mxfp4.h``): its records, its functions' types and the sizes.
Nothing here needs torch.
"""
from __future__ import annotations

import ctypes

import nvfp4_block_scaled_swiglu_amd as nv

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int


class _CCache(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("num_pages", _I64),
                ("page_size", _I64), ("kv_heads", _I64), ("head_dim", _I64)]


class _CBatch(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_lens", _P), ("cu_seqlens", _P), ("batch", _I64), ("max_pages", _I64),
                ("table_stride", _I64), ("tokens", _I64)]


class _CPrefix(ctypes.Structure):
    _fields_ = [("block_table", _P), ("lens", _P), ("group_starts", _P), ("groups", _I64), ("max_pages", _I64),
                ("table_stride", _I64)]


class _CNorm(ctypes.Structure):
    _fields_ = [("weight", _P), ("eps", ctypes.c_double)]


class _CRotation(ctypes.Structure):
    _fields_ = [("freqs", _P), ("axes_dev", _P), ("positions", _P), ("rotary_dim", _I64), ("axes", _I64),
                ("token_stride", _I64), ("axis_stride", _I64), ("interleaved", _INT)]


class _CPages(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_lens", _P), ("refs", _P), ("slots", _I64), ("max_pages", _I64),
                ("table_stride", _I64), ("num_pages", _I64), ("page_size", _I64)]


_PC = ctypes.POINTER(_CCache)
_PB = ctypes.POINTER(_CBatch)
_PX = ctypes.POINTER(_CPrefix)
_PN = ctypes.POINTER(_CNorm)
_PR = ctypes.POINTER(_CRotation)
_PP = ctypes.POINTER(_CPages)

# Every symbol include/mxfp4.h declares, with (restype, argtypes).
SIGNATURES = {
    "mxfp4_qdata_bytes": (_I64, [_I64, _I64]),
    "mxfp4_scale_cols": (_I64, [_I64]),
    "mxfp4_scale_bytes": (_I64, [_I64, _I64]),
    "mxfp4_quantize": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp4_quantize_swiglu": (_INT, [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp4_dequantize": (_INT, [_P, _P, _I64, _I64, _P, _I64, _P]),
    "mxfp4_gemm_bf16out": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "mxfp4_cache_append": (_INT, [_PC, _PB, _P, _I64, _I64, _P, _I64, _I64, _P]),
    "mxfp4_cache_read": (_INT, [_PC, _PB, _P, _I64, _I64, _P, _I64, _I64, _P]),
    "mxfp4_attention_workspace_bytes": (_I64, [_PC, _PB, _I64, _I64, _I64, _I64]),
    "mxfp4_attention": (_INT, [_PC, _PB, _P, _I64, _I64, _I64, ctypes.c_float, _INT, _I64, _I64, _I64, _P, _I64, _I64,
                               _P, _I64, _P]),
    "mxfp4_attention_prefix_workspace_bytes": (_I64, [_PC, _PB, _PX, _I64, _I64, _I64]),
    "mxfp4_attention_prefix": (_INT, [_PC, _PB, _PX, _P, _I64, _I64, _I64, ctypes.c_float, _INT, _I64, _I64, _P, _I64,
                                      _I64, _P, _I64, _P]),
    "mxfp4_norm_rope": (_INT, [_P, _I64, _I64, _I64, _I64, _I64, _PN, _PR, _P, _I64, _I64, _P]),
    "mxfp4_norm_rope_append": (_INT, [_PC, _PB, _P, _I64, _I64, _I64, _PN, _P, _I64, _I64, _PN, _P, _I64, _I64, _PR, _P,
                                      _I64, _I64, _P]),
    "mxfp4_pages_free": (_INT, [_PP, _P, _P, _I64, _P]),
    "mxfp4_pages_fork": (_INT, [_PP, _P, _P, _I64, _P, _P]),
    "mxfp4_pages_reserve_workspace_bytes": (_I64, [_PP, _I64]),
    "mxfp4_pages_reserve": (_INT, [_PP, _P, _P, _I64, _P, _P, _P, _P, _I64, _P]),
    "mxfp4_pages_compact_workspace_bytes": (_I64, [_PP]),
    "mxfp4_pages_compact": (_INT, [_PP, _P, _I64, _P, _P, _P, _P, _P, _I64, _P]),
    "mxfp4_cache_copy": (_INT, [_PC, _PC, _P, _P, _I64, _P]),
}


# ---- sizes ---------------------------------------------------------------------------------

def mxfp4_qdata_bytes(rows: int, k: int) -> int:
    return int(nv.lib().mxfp4_qdata_bytes(rows, k))


def mxfp4_scale_cols(k: int) -> int:
    return int(nv.lib().mxfp4_scale_cols(k))


def mxfp4_scale_bytes(rows: int, k: int) -> int:
    return int(nv.lib().mxfp4_scale_bytes(rows, k))
