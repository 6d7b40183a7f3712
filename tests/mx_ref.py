"""Plain statements of the MXFP4 operators in numpy / torch float64, for the tests: the format
from its definition (search among the eight magnitudes), the scale layout as reshapes, and
attention row by row. Shares no code with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bits_to_f64(bits: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bits(x: np.ndarray) -> np.ndarray:
    """float64 -> bf16 bits, one rounding, ties to even (finite results)."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    quantum = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    r = np.rint(x / quantum) * quantum
    r = np.where(r == 0.0, np.copysign(0.0, x), r)
    return (r.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def quantize(bits: np.ndarray):
    """bf16 bits [..., k] -> (codes uint8 [..., k/2], scale bytes uint8 [..., k/32])."""
    k = bits.shape[-1]
    x = bits_to_f64(bits).reshape(-1, BLOCK)
    finite = np.isfinite(x).all(1)
    x = np.where(finite[:, None], x, 0.0)
    top = np.abs(x).max(1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1, -1000)  # floor(log2 top)
    scale = np.where(finite, np.maximum(e - 2 + 127, 0), 255).astype(np.int64)
    y = np.abs(x) / np.ldexp(1.0, np.where(finite, scale - 127, 0))[:, None]
    dist = np.abs(np.minimum(y, 6.0)[:, :, None] - MAGNITUDES)
    best = dist.min(2, keepdims=True)
    # of the (at most two) nearest magnitudes the one with the even code
    rank = np.where(dist == best, np.arange(8) % 2, 2)
    code = rank.argmin(2)
    sign = (bits.reshape(-1, BLOCK) >> 15).astype(np.int64)
    code = np.where(finite[:, None], code + 8 * sign, 0).astype(np.uint8).reshape(-1, BLOCK // 2, 2)
    codes = code[:, :, 0] | (code[:, :, 1] << 4)
    lead = bits.shape[:-1]
    return codes.reshape(lead + (k // 2,)).astype(np.uint8), scale.astype(np.uint8).reshape(lead + (k // BLOCK,))


def values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """What codes and scale bytes stand for, float64 (NaN under byte 255)."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (codes.shape[-1] * 2,))
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, -1)


def round_trip(bits: np.ndarray) -> np.ndarray:
    return values(*quantize(bits))


def tiled(scale: np.ndarray) -> np.ndarray:
    """Scale bytes [rows, k/32] in storage order: 128 x 4 tiles, in a tile row r % 32, then
    r / 32, then the column; zero outside."""
    rows, cols = scale.shape
    pad = np.zeros((-(-rows // 128) * 128, -(-cols // 4) * 4), np.uint8)
    pad[:rows, :cols] = scale
    t = pad.reshape(pad.shape[0] // 128, 4, 32, pad.shape[1] // 4, 4)  # tile, r / 32, r % 32, group, column
    return t.transpose(0, 3, 2, 1, 4).reshape(-1)


def product(a: np.ndarray, w: np.ndarray):
    """(a @ w.T, |a| @ |w|.T) in float64."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def product_tolerance(ref: np.ndarray, mags: np.ndarray, k: int) -> np.ndarray:
    """|D - ref| of exact products, fp32 sums and one bf16 rounding. A matrix instruction adds 64
    or more products to the sum at a time: at most k / 64 + 1 additions in a chain and a few
    (waves') sums, each within 2^-23 of the magnitudes' sum, and inside an instruction at most 64
    more per product. The rounding is half a bf16 step: 2^-8 of the value, or 2^-134."""
    return (k / 64 + 80) * 2.0 ** -23 * mags + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133


def attention(q, k, v, scale, causal=True, window=0, sinks=0, hidden=None):
    """float64 torch tensors q [n, h, d], k, v [t, hk, d] -> (o, tolerance), both [n, h, d].

    hidden: bool [t], tokens that no row sees. The tolerance of o_d = sum_t w_t v_td against the
    library's arithmetic: scores are fp32 sums of exact products (d + 2 roundings of 2^-23 of
    sum |q||k|), which moves weights by that much, relatively, twice (numerator and sum); the
    weights are rounded to bf16, w_t (1 + e_t) with |e_t| <= 2^-8, for the product and for their
    sum: sum w (1 + e) v / sum w (1 + e) - o = sum w e (v - o) / sum w (1 + e), at most
    2^-8 (sum w |v| + |o|) beside terms of 2^-16; exp2, its argument and the fp32 sums over t
    stay within 2^-15, those terms with them within 2^-14 (arguments up to 2^6 in fp32: 2^-18,
    thousands of additions with 2^-24 each); the output is rounded once (2^-8). A weight below
    the smallest normal fp32 number
    may become 0: an error of at most 2^-126 beside a sum of weights of at least 1 (the running
    maximum never exceeds the largest score, whose weight is then at least 1), so at most
    2^-126 |v_td| of each token, and as much again for a product of o that falls below it."""
    import torch
    n, h, d = q.shape
    t, hk, _ = k.shape
    g = h // hk
    o = torch.zeros(n, h, d, dtype=torch.float64)
    tol = torch.zeros(n, h, d, dtype=torch.float64)
    for i in range(n):
        p = t - n + i
        at = torch.arange(t)
        seen = torch.ones(t, dtype=torch.bool)
        if causal:
            seen &= at <= p
        if window:
            seen &= (at > p - window) | (at < sinks)
        if hidden is not None:
            seen &= ~hidden
        if not bool(seen.any()):
            continue
        for j in range(h):
            kk, vv = k[seen, j // g], v[seen, j // g]
            s = kk @ q[i, j] * scale
            mag = float((kk.abs() @ q[i, j].abs() * scale).max())
            w = torch.softmax(s, 0)
            o[i, j] = w @ vv
            err = 2.0 ** -8 + 2.0 ** -14 + 2 * (d + 2) * 2.0 ** -23 * mag
            tiny = 2.0 ** -126 * (vv.abs().sum(0) + vv.shape[0])
            tol[i, j] = err * (w @ vv.abs()) + 2 * 2.0 ** -8 * o[i, j].abs() + tiny
    return o, tol
