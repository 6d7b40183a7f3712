"""Norms and rotation of query and key heads (``include/mxfp4.h``) - Python binding.

``mxfp4_norm_rope(x)`` gives bf16 heads back, ``mxfp4_norm_rope_append(cache, q, k, v, ...)`` does
all that stands between a QKV projection and ``mxfp4_attention`` in one launch. Calls, checks,
streams and errors are those of ``mxfp4.py``.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Sequence

import torch

import nvfp4_block_scaled_swiglu_amd as nv

from .mxfp4 import (Mxfp4Cache, _batch, _bf16, _cache, _CNorm, _CRotation, _On, _strides, _Tensor)


@dataclass
class Mxfp4Rotation:
    """What turns the pairs of a head: of the first 2 * len(freqs) elements, pair j - elements
    (j, j + len(freqs)), interleaved (2 j, 2 j + 1) - turns by freqs[j] radians for each step of
    the position on axis axes[j]."""
    freqs: torch.Tensor                    # float32 [rotary_dim / 2]
    axes: Optional[torch.Tensor] = None    # int32 [rotary_dim / 2]; None: axis 0
    axis_count: int = 1
    interleaved: bool = False


def mxfp4_rotation(rotary_dim: int, device, theta: float = 10000.0, sections: Optional[Sequence[int]] = None,
                   separate: bool = False, interleaved: bool = False) -> Mxfp4Rotation:
    """The usual frequencies theta ** (-2 j / rotary_dim). sections: how many pairs each axis has, in
    order (a time, height and width axis, say; they add up to rotary_dim / 2); separate: the
    frequencies of an axis then run over its own pairs, theta ** (-i / pairs), i from 0."""
    pairs = rotary_dim // 2
    sections = [pairs] if sections is None else [int(n) for n in sections]
    if rotary_dim <= 0 or rotary_dim % 2 or not sections or min(sections) < 0 or sum(sections) != pairs:
        raise ValueError("sections must add up to rotary_dim / 2")
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    exponents = [i / n for n in sections for i in range(n)] if separate else [j / pairs for j in range(pairs)]
    return Mxfp4Rotation(torch.tensor([theta ** -e for e in exponents], dtype=torch.float32, device=device),
                         torch.tensor(axes, dtype=torch.int32, device=device) if len(sections) > 1 else None,
                         len(sections), interleaved)


def _vector(t, name: str, dtype, size: Optional[int] = None):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != 1 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D {str(dtype).split('.')[-1]} CUDA tensor")
    if size is not None and t.shape[0] != size:
        raise ValueError(f"{name} must have {size} elements, not {t.shape[0]}")
    return t


def _rotation(rotation: Optional[Mxfp4Rotation], positions, tokens: int, dim: int, cached: bool):
    """The rotation's C form and its tensors."""
    if rotation is None:
        if positions is not None:
            raise ValueError("positions without a rotation")
        return None, ()
    if not isinstance(rotation, Mxfp4Rotation):
        raise ValueError("rotation must be an Mxfp4Rotation")
    pairs = _vector(rotation.freqs, "rotation.freqs", torch.float32).shape[0]
    tensors = [rotation.freqs]
    if rotation.axes is not None:
        tensors.append(_vector(rotation.axes, "rotation.axes", torch.int32, pairs))
    if not 1 <= rotation.axis_count <= 64:
        raise ValueError("rotation.axis_count must be 1 to 64")
    token_stride = axis_stride = 0
    if positions is None:
        if not cached:
            raise ValueError("positions are needed where there is no cache")
    else:
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32 or not positions.is_cuda:
            raise ValueError("positions must be an int32 CUDA tensor")
        if positions.shape != (tokens,) and positions.shape != (tokens, rotation.axis_count):
            raise ValueError(f"positions must have shape {(tokens,)} or {(tokens, rotation.axis_count)}, "
                             f"not {tuple(positions.shape)}")
        token_stride = positions.stride(0) if tokens > 1 else 0
        axis_stride = positions.stride(1) if positions.dim() == 2 and rotation.axis_count > 1 else 0
        tensors.append(positions)
    return _CRotation(rotation.freqs.data_ptr(), None if rotation.axes is None else rotation.axes.data_ptr(),
                      None if positions is None else positions.data_ptr(), 2 * pairs, rotation.axis_count, token_stride,
                      axis_stride, int(bool(rotation.interleaved))), tensors


def _norm(weight, eps: Optional[float], name: str, dim: int):
    """The norm's C form and its tensors."""
    if eps is None:
        if weight is not None:
            raise ValueError(f"{name} without eps")
        return None, ()
    if weight is None:
        return _CNorm(None, eps), ()
    _vector(weight, name, torch.bfloat16, dim)
    return _CNorm(weight.data_ptr(), eps), (weight,)


def mxfp4_norm_rope(x, rotation: Optional[Mxfp4Rotation] = None, positions=None, weight=None, eps: Optional[float] = None,
                    out=None, stream=None, strict: Optional[bool] = None):
    """Heads x (bf16 [tokens, heads, head_dim of 64, 128 or 256]) normed over head_dim (eps: not
    None; weight: bf16 [head_dim], or None for ones) and rotated at positions (int32 [tokens], or
    [tokens, axes] with one on each of the rotation's axes). out may be x."""
    tokens, heads, dim = _bf16(x, "x", 3).shape
    r, rt = _rotation(rotation, positions, tokens, dim, False)
    n, nt = _norm(weight, eps, "weight", dim)
    with _On(stream, x, *rt, *nt) as on:
        if out is None:
            out = x.new_empty((tokens, heads, dim))
        elif _bf16(out, "out", 3, x.shape).device != on.device:
            raise ValueError("out must be on the device of x")
        else:
            on.use(out)
        if not nv._call("mxfp4_norm_rope", x.data_ptr(), *_strides(x), tokens, heads, dim, n, r, out.data_ptr(),
                        *_strides(out), on.handle, strict=strict):
            return None
    return out


def mxfp4_norm_rope_append(cache: Mxfp4Cache, q, k, v, block_table, seq_lens, cu_seqlens,
                           rotation: Optional[Mxfp4Rotation] = None, positions=None, q_weight=None, k_weight=None,
                           eps: Optional[float] = None, out=None, stream=None, strict: Optional[bool] = None):
    """q, k and v of new tokens (bf16 [tokens, heads or kv_heads, head_dim]) on their way from the
    projection: q and k normed (eps: not None) and rotated, k and v quantized into the cache at their
    rows' positions as mxfp4_cache_append does. Returns q's new values (out, which may be q).

    positions: as in mxfp4_norm_rope; by default the rows' positions in their sequences. Rows
    behind the last sequence keep what out held."""
    c, ct = _cache(cache)
    tokens, heads, dim = _bf16(q, "q", 3).shape
    if dim != c.head_dim:
        raise ValueError(f"q has head_dim {dim}, the cache {c.head_dim}")
    shape = (tokens, c.kv_heads, dim)
    _bf16(k, "k", 3, shape)
    _bf16(v, "v", 3, shape)
    b, bt = _batch(block_table, seq_lens, cu_seqlens, tokens)
    r, rt = _rotation(rotation, positions, tokens, dim, True)
    qn, qt = _norm(q_weight, eps, "q_weight", dim)
    kn, kt = _norm(k_weight, eps, "k_weight", dim)
    with _On(stream, q, k, v, *ct, *bt, *rt, *qt, *kt) as on:
        if out is None:
            out = q.new_empty((tokens, heads, dim))
        elif _bf16(out, "out", 3, q.shape).device != on.device:
            raise ValueError("out must be on the device of q")
        else:
            on.use(out)
        if not nv._call("mxfp4_norm_rope_append", c, b, q.data_ptr(), *_strides(q), heads, qn, k.data_ptr(), *_strides(k), kn,
                        v.data_ptr(), *_strides(v), r, out.data_ptr(), *_strides(out), on.handle, strict=strict):
            return None
    return out
