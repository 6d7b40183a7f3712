"""MXFP4 operators of the library (``include/mxfp4.h``) - Python binding.

MXFP4 is the 4-bit format with one power-of-two scale per 32 elements that gfx950's scaled
matrix instructions multiply as it is stored. Functions carry the C names:

* ``mxfp4_quantize(x)``, ``mxfp4_quantize_swiglu(gate, up)`` - bf16 -> MXFP4, one pass
* ``mxfp4_dequantize(t)``                                    - and back
* ``mxfp4_gemm_bf16out(a, w)``                               - product of two, BF16 out, from one row up
* ``mxfp4_cache_append(...)``, ``mxfp4_cache_read(...)``     - a paged key/value cache in MXFP4
* ``mxfp4_attention(q, cache, ...)``                         - attention over that cache
* ``mxfp4_attention_prefix(q, cache, ...)``                  - where groups of sequences share their first pages
* ``mxfp4_norm_rope(x, ...)``, ``mxfp4_norm_rope_append(...)`` - head norms and rotation, and on into the cache
  (``mxfp4_rope.py``)
* ``mxfp4_pages_*(...)``, ``mxfp4_cache_copy(...)``           - which pages the sequences hold (``mxfp4_pages.py``)

As elsewhere in the package every step runs in the library's kernels, a failing call raises
(strict) or returns None and counts a fallback, and outputs that the caller does not pass are
allocated with torch. Calls run on the device of their tensors (which must be one) and on
``stream``, by default that device's current stream; with another stream given, outputs and
workspaces are allocated for it, and the tensors that the caller passes (inputs, outputs and
workspaces) are marked as used by it.

A packed batch is described by ``block_table`` (int32 [batch, max_pages]: page numbers),
``seq_lens`` (int32 [batch]: cached tokens of each sequence, the call's new ones included) and
``cu_seqlens`` (int32 [batch + 1]: first row of each sequence in the packed tensors, from 0):
the rows of a sequence are the last tokens of its cache. Page numbers out of range and rows
behind the last sequence are skipped; rows behind the last sequence keep what the output held.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

import nvfp4_block_scaled_swiglu_amd as nv

from .mxfp4_abi import (  # noqa: F401  (the C side, by its names here too)
    SIGNATURES, _CBatch, _CCache, _CNorm, _CPages, _CPrefix, _CRotation, mxfp4_qdata_bytes, mxfp4_scale_bytes,
    mxfp4_scale_cols)


# ---- tensors -------------------------------------------------------------------------------

@dataclass
class Mxfp4Tensor:
    """A quantized [rows, k] tensor as the library lays it out in device memory."""
    qdata: torch.Tensor   # uint8 [rows, k/2]
    scales: torch.Tensor  # uint8 [mxfp4_scale_bytes(rows, k)], 128x4-tiled
    rows: int
    k: int


@dataclass
class Mxfp4Cache:
    """A paged key/value cache: per page and kv head, page_size rows of codes and scales."""
    k_codes: torch.Tensor   # uint8 [num_pages, kv_heads, page_size, head_dim / 2]
    k_scales: torch.Tensor  # uint8 [num_pages, kv_heads, page_size, head_dim / 32]
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    @property
    def num_pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k_codes.shape[3] * 2


def empty_mxfp4(rows: int, k: int, device) -> Mxfp4Tensor:
    return Mxfp4Tensor(qdata=torch.empty((rows, k // 2), dtype=torch.uint8, device=device),
                       scales=torch.empty((max(0, _scale_bytes(rows, k)),), dtype=torch.uint8, device=device),
                       rows=rows, k=k)


def empty_mxfp4_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, device) -> Mxfp4Cache:
    """A cache whose contents are undefined until they are appended."""
    shape = (num_pages, kv_heads, page_size)
    make = lambda n: torch.empty(shape + (n,), dtype=torch.uint8, device=device)  # noqa: E731
    return Mxfp4Cache(make(head_dim // 2), make(head_dim // 32), make(head_dim // 2), make(head_dim // 32))


# ---- checks and streams --------------------------------------------------------------------

# A small call is as long as its checks: names of this module are found faster than torch's. (A token into the
# cache through mxfp4_norm_rope_append 14.2 -> 13.3 us, its read 12.2 -> 10.)
_Tensor, _BF16, _INT32, _UINT8 = torch.Tensor, torch.bfloat16, torch.int32, torch.uint8
_device_of = torch.Tensor.get_device


def _bf16(t, name: str, dim: int, shape=None):
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.dim() != dim or not t.is_cuda:
        raise ValueError(f"{name} must be a {dim}-D bfloat16 CUDA tensor")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t


def _buffer(t, name: str, size: int):
    if not isinstance(t, _Tensor) or t.dtype is not _UINT8 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
    if t.numel() < size:
        raise ValueError(f"{name} holds {t.numel()} bytes, {size} needed")
    return t


_MOST = (1 << 63) - 1  # larger numbers are cut to 64 bits on their way into the library


def _packed(t, name: str):
    if not isinstance(t, Mxfp4Tensor):
        raise ValueError(f"{name} must be an Mxfp4Tensor")
    if t.rows < -_MOST or t.k < -_MOST:  # (if larger than _MOST the buffers are too small)
        raise ValueError(f"{name}.rows and k must fit 64 bits")
    _buffer(t.qdata, name, t.rows * (t.k // 2))
    _buffer(t.scales, name, _scale_bytes(t.rows, t.k))
    return t


def _scale_bytes(rows: int, k: int) -> int:  # mxfp4_scale_bytes without the call
    return -(-rows // 128) * 128 * (-(-(k // 32) // 4) * 4)


def _int32(t, name: str, dim: int):
    if not isinstance(t, _Tensor) or t.dtype is not _INT32 or t.dim() != dim or not t.is_cuda:
        raise ValueError(f"{name} must be a {dim}-D int32 CUDA tensor")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return t


def _row_stride(t) -> int:
    """Row stride of a 2-D tensor; of a single row, whose stride means nothing, its length
    rounded up to the 8 elements that the library asks for."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _strides(t) -> Tuple[int, int]:
    """(token, head) strides of [tokens, heads, dim]; those of single ones mean nothing."""
    shape, strides = t.shape, t.stride()
    return (strides[0] if shape[0] > 1 else 0, strides[1] if shape[1] > 1 else shape[2])


def _stream_object(index: int) -> int:
    return int(torch.cuda.current_stream(index).cuda_stream)


# The current device, and the handle of its current stream without the object around it, where torch has them so.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_object)


class _On:
    """The device and stream of a call: enter it to allocate outputs and to launch."""

    __slots__ = ("device", "handle", "stack", "side")

    def __init__(self, stream, *tensors):
        devices = set(map(_device_of, tensors))
        if len(devices) != 1:
            raise ValueError("all tensors of a call must be on one device")
        index, = devices
        self.device = tensors[0].device
        self.stack = self.side = None
        if stream is None and index == _current_device():  # nothing to switch
            self.handle = _current_stream(index)
            return
        self.stack = contextlib.ExitStack()
        try:
            self.stack.enter_context(torch.cuda.device(self.device))
            current = torch.cuda.current_stream()
            if stream is not None and stream != current:
                if getattr(stream, "device", self.device) != self.device:
                    raise ValueError("stream is of another device than the tensors")
                self.stack.enter_context(torch.cuda.stream(stream))
                self.side = current = stream
                self.use(*tensors)
            self.handle = int(current.cuda_stream)
        except BaseException:
            self.stack.close()
            raise

    def use(self, *tensors):
        """Marks the caller's tensors as used by the call's stream if that is not the current one."""
        if self.side is not None:
            for t in tensors:
                t.record_stream(self.side)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self.stack is not None:
            return self.stack.__exit__(*exc)


# ---- quantization --------------------------------------------------------------------------

def _quantize_out(on: _On, out, rows: int, k: int):
    device = on.device
    if out is None:
        return empty_mxfp4(rows, k, device)
    _packed(out, "out")
    if out.rows != rows or out.k != k or out.qdata.device != device or out.scales.device != device:
        raise ValueError("out must be an Mxfp4Tensor for the same rows and k on the same device")
    on.use(out.qdata, out.scales)
    return out


def mxfp4_quantize(x, out: Optional[Mxfp4Tensor] = None, stream=None,
                   strict: Optional[bool] = None) -> Optional[Mxfp4Tensor]:
    """MXFP4 of a bf16 [rows, k] tensor (k a multiple of 32): codes and 128x4-tiled scales."""
    _bf16(x, "x", 2)
    rows, k = x.shape
    with _On(stream, x) as on:
        out = _quantize_out(on, out, rows, k)
        if not nv._call("mxfp4_quantize", x.data_ptr(), _row_stride(x), rows, k, out.qdata.data_ptr(),
                        out.scales.data_ptr(), on.handle, strict=strict):
            return None
    return out


def mxfp4_quantize_swiglu(gate, up, out: Optional[Mxfp4Tensor] = None, stream=None,
                          strict: Optional[bool] = None) -> Optional[Mxfp4Tensor]:
    """MXFP4 of y = RN_bf16(silu_bf16(gate) * up), the y of nvfp4_quantize_swiglu."""
    _bf16(gate, "gate", 2)
    _bf16(up, "up", 2, gate.shape)
    m, k = gate.shape
    with _On(stream, gate, up) as on:
        out = _quantize_out(on, out, m, k)
        if not nv._call("mxfp4_quantize_swiglu", gate.data_ptr(), _row_stride(gate), up.data_ptr(), _row_stride(up), m, k,
                        out.qdata.data_ptr(), out.scales.data_ptr(), on.handle, strict=strict):
            return None
    return out


def mxfp4_dequantize(t: Mxfp4Tensor, out=None, stream=None, strict: Optional[bool] = None):
    """The bf16 [rows, k] values of a quantized tensor (exact)."""
    _packed(t, "t")
    with _On(stream, t.qdata, t.scales) as on:
        if out is None:
            out = torch.empty((t.rows, t.k), dtype=torch.bfloat16, device=on.device)
        elif _bf16(out, "out", 2, (t.rows, t.k)).device != on.device:
            raise ValueError("out must be on the device of t")
        else:
            on.use(out)
        if not nv._call("mxfp4_dequantize", t.qdata.data_ptr(), t.scales.data_ptr(), t.rows, t.k, out.data_ptr(),
                        _row_stride(out), on.handle, strict=strict):
            return None
    return out


# ---- product -------------------------------------------------------------------------------

def mxfp4_gemm_bf16out(a: Mxfp4Tensor, w: Mxfp4Tensor, out=None, stream=None, strict: Optional[bool] = None):
    """D[m, n] = RN_bf16(sum_k A[m, k] W[n, k]) of a [m, k] and w [n, k], FP32 accumulation."""
    _packed(a, "a")
    _packed(w, "w")
    if a.k != w.k:
        raise ValueError("k mismatch")
    m, n = a.rows, w.rows
    with _On(stream, a.qdata, a.scales, w.qdata, w.scales) as on:
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=on.device)
        elif _bf16(out, "out", 2, (m, n)).device != on.device:
            raise ValueError("out must be on the device of a and w")
        else:
            on.use(out)
        if not nv._call("mxfp4_gemm_bf16out", a.qdata.data_ptr(), a.scales.data_ptr(), w.qdata.data_ptr(),
                        w.scales.data_ptr(), out.data_ptr(), out.stride(0) if m > 1 else n, m, n, a.k, on.handle,
                        strict=strict):
            return None
    return out


# ---- paged cache and attention -------------------------------------------------------------

def _cache(c: Mxfp4Cache):
    """The cache's C form and its tensors."""
    if not isinstance(c, Mxfp4Cache):
        raise ValueError("cache must be an Mxfp4Cache")
    kc, ks, vc, vs = tensors = (c.k_codes, c.k_scales, c.v_codes, c.v_scales)
    for t in tensors:
        if not isinstance(t, _Tensor) or t.dtype is not _UINT8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("the cache's tensors must be contiguous uint8 CUDA tensors")
    if kc.dim() != 4:
        raise ValueError("cache.k_codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
    pages, heads, size, half = kc.shape
    scales = (pages, heads, size, half // 16)
    if vc.shape != kc.shape or ks.shape != scales or vs.shape != scales:
        raise ValueError("the cache's codes and scales disagree in shape")
    return _CCache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, size, heads, 2 * half), tensors


def _batch(block_table, seq_lens, cu_seqlens, tokens: int):
    _int32(block_table, "block_table", 2)
    _int32(seq_lens, "seq_lens", 1)
    _int32(cu_seqlens, "cu_seqlens", 1)
    batch, pages = block_table.shape
    if seq_lens.shape[0] != batch or cu_seqlens.shape[0] != batch + 1:
        raise ValueError("block_table, seq_lens and cu_seqlens disagree about the batch")
    stride = block_table.stride(0) if batch > 1 else pages
    return (_CBatch(block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), batch, pages, stride, tokens),
            (block_table, seq_lens, cu_seqlens))


def mxfp4_cache_append(cache: Mxfp4Cache, k, v, block_table, seq_lens, cu_seqlens, stream=None,
                       strict: Optional[bool] = None) -> Optional[Mxfp4Cache]:
    """Quantize new keys and values (bf16 [tokens, kv_heads, head_dim]) into the cache at their
    rows' positions, the last ones of each sequence. Returns the cache."""
    c, ct = _cache(cache)
    shape = _bf16(k, "k", 3).shape
    if shape[1] != c.kv_heads or shape[2] != c.head_dim:
        raise ValueError(f"k must have shape {(shape[0], c.kv_heads, c.head_dim)}, not {tuple(shape)}")
    _bf16(v, "v", 3, shape)
    b, bt = _batch(block_table, seq_lens, cu_seqlens, shape[0])
    with _On(stream, k, v, *ct, *bt) as on:
        if not nv._call("mxfp4_cache_append", c, b, k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), on.handle,
                        strict=strict):
            return None
    return cache


def mxfp4_cache_read(cache: Mxfp4Cache, block_table, seq_lens, cu_seqlens, tokens: int, out=None, stream=None,
                     strict: Optional[bool] = None):
    """(k, v), each bf16 [tokens, kv_heads, head_dim]: the values of the rows' positions, the
    last cu_seqlens[b + 1] - cu_seqlens[b] tokens of each sequence. out: such a pair."""
    c, ct = _cache(cache)
    b, bt = _batch(block_table, seq_lens, cu_seqlens, tokens)
    shape = (tokens, c.kv_heads, c.head_dim)
    with _On(stream, *ct, *bt) as on:
        if out is None:
            k = torch.empty(shape, dtype=torch.bfloat16, device=on.device)
            v = torch.empty_like(k)
        else:
            k, v = out
            if _bf16(k, "out k", 3, shape).device != on.device or _bf16(v, "out v", 3, shape).device != on.device:
                raise ValueError("out must be on the device of the cache")
            on.use(k, v)
        if not nv._call("mxfp4_cache_read", c, b, k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), on.handle,
                        strict=strict):
            return None
    return k, v


def _limits(max_kv: int, window: int, sinks: int):
    if not (-_MOST <= max_kv <= _MOST and -_MOST <= window <= _MOST and -_MOST <= sinks <= _MOST):
        raise ValueError("max_kv, window and sinks must fit 64 bits")


def mxfp4_attention(q, cache: Mxfp4Cache, block_table, seq_lens, cu_seqlens, scale: Optional[float] = None,
                    causal: bool = True, window: int = 0, sinks: int = 0, max_kv: Optional[int] = None, out=None,
                    workspace=None, stream=None, strict: Optional[bool] = None):
    """Attention of packed queries (bf16 [tokens, heads, head_dim]) over the cached tokens of
    their sequences; heads a multiple of the cache's kv_heads, which query heads share in order.

    causal: a row sees the tokens up to its own position. window > 0: of those only the last
    `window`, and the first `sinks` tokens. scale: up to 2^127, by default head_dim ** -0.5. max_kv: the
    longest cached length as far as known (by default what the block table could hold); it
    decides how the work is split. workspace: a uint8 tensor of at least
    mxfp4_attention_workspace_bytes(...) bytes, allocated by default. Rows that see nothing give
    zeros; rows behind the last sequence keep what out held."""
    c, ct = _cache(cache)
    _bf16(q, "q", 3)
    tokens, heads, dim = q.shape
    if dim != c.head_dim:
        raise ValueError(f"q has head_dim {dim}, the cache {c.head_dim}")
    b, bt = _batch(block_table, seq_lens, cu_seqlens, tokens)
    if scale is None:
        scale = dim ** -0.5
    if max_kv is None:
        max_kv = max(1, b.max_pages * c.page_size)
    _limits(max_kv, window, sinks)
    with _On(stream, q, *ct, *bt) as on:
        if out is None:
            out = q.new_empty((tokens, heads, dim))
        elif _bf16(out, "out", 3, q.shape).device != on.device:
            raise ValueError("out must be on the device of q")
        else:
            on.use(out)
        if workspace is None:
            size = nv.lib().mxfp4_attention_workspace_bytes(c, b, heads, max_kv, window, sinks)
            if size > 0:
                workspace = torch.empty((size,), dtype=torch.uint8, device=on.device)
        elif _buffer(workspace, "workspace", 0).device != on.device:
            raise ValueError("workspace must be on the device of q")
        else:
            on.use(workspace)
        if not nv._call("mxfp4_attention", c, b, q.data_ptr(), *_strides(q), heads, scale, int(bool(causal)), window, sinks,
                        max_kv, out.data_ptr(), *_strides(out), 0 if workspace is None else workspace.data_ptr(),
                        0 if workspace is None else workspace.numel(), on.handle, strict=strict):
            return None
    return out


def mxfp4_attention_workspace_bytes(cache: Mxfp4Cache, block_table, seq_lens, cu_seqlens, tokens: int, heads: int,
                                    max_kv: int, window: int = 0, sinks: int = 0) -> int:
    """Bytes of the workspace of a call of these sizes (0: none); raises ValueError where the
    call would be refused."""
    _limits(max_kv, window, sinks)
    if not (-_MOST <= tokens <= _MOST and -_MOST <= heads <= _MOST):
        raise ValueError("tokens and heads must fit 64 bits")
    c, _ = _cache(cache)
    b, _ = _batch(block_table, seq_lens, cu_seqlens, tokens)
    size = int(nv.lib().mxfp4_attention_workspace_bytes(c, b, heads, max_kv, window, sinks))
    if size < 0:
        raise ValueError(nv.lib().nvfp4_last_error().decode(errors="replace"))
    return size


# ---- attention behind shared prefixes ------------------------------------------------------

def _prefix(prefix_table, prefix_lens, group_starts):
    _int32(prefix_table, "prefix_table", 2)
    _int32(prefix_lens, "prefix_lens", 1)
    _int32(group_starts, "group_starts", 1)
    groups, pages = prefix_table.shape
    if prefix_lens.shape[0] != groups or group_starts.shape[0] != groups + 1:
        raise ValueError("prefix_table, prefix_lens and group_starts disagree about the groups")
    stride = prefix_table.stride(0) if groups > 1 else pages
    return (_CPrefix(prefix_table.data_ptr(), prefix_lens.data_ptr(), group_starts.data_ptr(), groups, pages, stride),
            (prefix_table, prefix_lens, group_starts))


def _most(given: Optional[int], pages: int, page_size: int) -> int:
    most = max(1, pages * page_size) if given is None else given
    if not -_MOST <= most <= _MOST:
        raise ValueError("max_prefix and max_own must fit 64 bits")
    return most


def mxfp4_attention_prefix(q, cache: Mxfp4Cache, block_table, seq_lens, cu_seqlens, prefix_table, prefix_lens, group_starts,
                           scale: Optional[float] = None, causal: bool = True, max_prefix: Optional[int] = None,
                           max_own: Optional[int] = None, out=None, workspace=None, stream=None,
                           strict: Optional[bool] = None):
    """mxfp4_attention (without a window) of sequences whose groups share their first tokens, which
    are then read once for a group.

    Group g is the sequences group_starts[g] .. group_starts[g + 1] - 1 (int32 [groups + 1],
    ascending); the first prefix_lens[g] // 64 * 64 of their tokens are those in the pages of
    prefix_table[g] (int32 [groups, max_pages]). Other tokens go by block_table, and so do all tokens of
    sequences in no group or whose first row does not see every shared token. max_prefix, max_own: the
    longest prefix, and the most tokens of a sequence behind its own, as far as known (by default
    what the tables could hold, which can take half as long again); they decide how the work is split. workspace: a uint8 tensor of at least
    mxfp4_attention_prefix_workspace_bytes(...) bytes, allocated by default."""
    c, ct = _cache(cache)
    _bf16(q, "q", 3)
    tokens, heads, dim = q.shape
    if dim != c.head_dim:
        raise ValueError(f"q has head_dim {dim}, the cache {c.head_dim}")
    b, bt = _batch(block_table, seq_lens, cu_seqlens, tokens)
    x, xt = _prefix(prefix_table, prefix_lens, group_starts)
    if scale is None:
        scale = dim ** -0.5
    max_prefix, max_own = _most(max_prefix, x.max_pages, c.page_size), _most(max_own, b.max_pages, c.page_size)
    with _On(stream, q, *ct, *bt, *xt) as on:
        if out is None:
            out = q.new_empty((tokens, heads, dim))
        elif _bf16(out, "out", 3, q.shape).device != on.device:
            raise ValueError("out must be on the device of q")
        else:
            on.use(out)
        if workspace is None:
            size = nv.lib().mxfp4_attention_prefix_workspace_bytes(c, b, x, heads, max_prefix, max_own)
            if size > 0:
                workspace = torch.empty((size,), dtype=torch.uint8, device=on.device)
        elif _buffer(workspace, "workspace", 0).device != on.device:
            raise ValueError("workspace must be on the device of q")
        else:
            on.use(workspace)
        if not nv._call("mxfp4_attention_prefix", c, b, x, q.data_ptr(), *_strides(q), heads, scale, int(bool(causal)),
                        max_prefix, max_own, out.data_ptr(), *_strides(out), 0 if workspace is None else workspace.data_ptr(),
                        0 if workspace is None else workspace.numel(), on.handle, strict=strict):
            return None
    return out


def mxfp4_attention_prefix_workspace_bytes(cache: Mxfp4Cache, block_table, seq_lens, cu_seqlens, prefix_table, prefix_lens,
                                           group_starts, tokens: int, heads: int, max_prefix: Optional[int] = None,
                                           max_own: Optional[int] = None) -> int:
    """Bytes of the workspace of a call of these sizes; raises ValueError where the call would be refused."""
    if not (-_MOST <= tokens <= _MOST and -_MOST <= heads <= _MOST):
        raise ValueError("tokens and heads must fit 64 bits")
    c, _ = _cache(cache)
    b, _ = _batch(block_table, seq_lens, cu_seqlens, tokens)
    x, _ = _prefix(prefix_table, prefix_lens, group_starts)
    size = int(nv.lib().mxfp4_attention_prefix_workspace_bytes(
        c, b, x, heads, _most(max_prefix, x.max_pages, c.page_size), _most(max_own, b.max_pages, c.page_size)))
    if size < 0:
        raise ValueError(nv.lib().nvfp4_last_error().decode(errors="replace"))
    return size
