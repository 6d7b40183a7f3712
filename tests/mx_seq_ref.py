"""Plain statements, for the tests, of what surrounds the MXFP4 cache: norms and rotation in numpy
float64 with angles from exact rationals, and the pages' bookkeeping as lists. Shares no code with
the library."""
from __future__ import annotations

from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np

getcontext().prec = 70
TWO_PI = 2 * Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"))


def turns(positions: np.ndarray, freqs: np.ndarray, axes=None) -> np.ndarray:
    """angles [tokens, pairs] as float64 radians in [-pi, pi], from the exact product: positions
    int [tokens, axis count], freqs float32 [pairs], axes [pairs]."""
    out = np.zeros((positions.shape[0], freqs.shape[0]))
    for j, f in enumerate(freqs):
        step = Fraction(float(f)) / TWO_PI
        for i in range(positions.shape[0]):
            t = step * int(positions[i, 0 if axes is None else axes[j]])
            out[i, j] = float((t - round(t)) * TWO_PI)
    return out


def norm_rope(x: np.ndarray, angle=None, interleaved=False, eps=None, weight=None):
    """float64 [tokens, heads, dim] -> (y, size): the result and the magnitude that its last sum's
    rounding goes by (|a cos| + |b sin|)."""
    y = np.array(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if eps is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
            if weight is not None:
                y = y * weight
        size = np.abs(y)
        if angle is not None:
            r = 2 * angle.shape[1]
            first = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
            second = first + (1 if interleaved else r // 2)
            c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
            a, b = y[..., first].copy(), y[..., second].copy()
            y[..., first], y[..., second] = a * c - b * s, b * c + a * s
            size[..., first], size[..., second] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, size


def norm_rope_tolerance(y: np.ndarray, size: np.ndarray) -> np.ndarray:
    """Of the fp32 form. The sum of squares: a chain of 16 and up to 4 more additions of positive
    terms, 20 roundings of 2^-24, and 3 more for the mean and eps; under the root half of them, then the
    root, the reciprocal and the two products: under 18 x 2^-24 of the normed value. Cosine and sine
    rounded to fp32, a product and an fma: 3 more, of |a cos| + |b sin|. 21 x 2^-24 < 2^-19 of `size`. Then one
    rounding to bf16, 2^-8 of the value, or half of the smallest number, 2^-134; and fp32's own smallest
    normal number where a product falls below it."""
    fine = 2.0 ** -19 * size
    return fine + 2.0 ** -8 * (np.abs(y) + fine) + 2.0 ** -125


class Pages:
    """The bookkeeping, one step at a time."""

    def __init__(self, slots, max_pages, num_pages, page):
        self.table = np.full((slots, max_pages), -1, np.int64)
        self.lens = np.zeros(slots, np.int64)
        self.refs = np.zeros(num_pages, np.int64)
        self.page = page

    def held(self, n):
        return min(-(-n // self.page), self.table.shape[1])

    def free(self, slots, keep=None):
        for i, s in enumerate(slots):
            if not 0 <= s < len(self.lens):
                continue
            k = 0 if keep is None else max(0, keep[i])
            if k >= self.lens[s]:
                continue
            for e in range(self.held(k), self.held(self.lens[s])):
                self.refs[self.table[s, e]] -= 1
                self.table[s, e] = -1
            self.lens[s] = k

    def fork(self, parents, children):
        before = self.lens.copy()
        done = []
        for i, (p, c) in enumerate(zip(parents, children)):
            ok = 0 <= p < len(before) and 0 <= c < len(before) and c not in children[:i] and p not in children \
                and before[c] == 0
            done.append(int(ok))
            if ok:
                n = self.held(before[p])
                self.table[c, :n] = self.table[p, :n]
                self.lens[c] = before[p]
                for e in range(n):
                    self.refs[self.table[p, e]] += 1
        return done

    def reserve(self, slots, lens):
        refs = self.refs.copy()
        free = [p for p in range(len(refs)) if refs[p] < 1]
        at, done, src, dst = 0, [], [], []
        for i, (s, n) in enumerate(zip(slots, lens)):
            done.append(0), src.append(-1), dst.append(-1)
            if not 0 <= s < len(self.lens) or s in slots[:i] or n < self.lens[s] or n > self.table.shape[1] * self.page:
                continue
            old, have = self.lens[s], self.held(self.lens[s])
            last = self.table[s, have - 1] if have else -1
            copies = n > old and old % self.page != 0 and refs[last] > 1
            need = self.held(n) - have + copies
            start, at = at, at + need
            if need and at > len(free):
                continue
            new = free[start:at]
            done[-1] = 1
            if copies:
                src[-1], dst[-1] = last, new[0]
                self.refs[last] -= 1
            for k, p in enumerate(new):
                self.table[s, have - copies + k] = p
                self.refs[p] = 1
            self.lens[s] = n
        return done, src, dst

    def compact(self):
        used = int((self.refs > 0).sum())
        src = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] < 1]
        to = dict(zip(src, dst))
        for s in range(len(self.lens)):
            for e in range(self.held(self.lens[s])):
                self.table[s, e] = to.get(self.table[s, e], self.table[s, e])
        refs = np.where(self.refs > 0, self.refs, 0)
        for a, b in to.items():
            refs[b], refs[a] = refs[a], 0
        self.refs = refs
        pad = [-1] * (len(self.refs) // 2 - len(src))
        return src + pad, dst + pad, used
