"""Oracle of the 8-bit cache in float64: what a sequence's blocks hold after tokens were
appended in parts, and the record's bytes.  TEST INFRASTRUCTURE ONLY (see the package header)."""

from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def e4m3_value(code):
    e, m = (code >> 3) & 15, code & 7
    if (code & 127) == 127:
        return math.nan
    x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -x if code & 128 else x


E4M3 = np.array([e4m3_value(c) for c in range(256)])
_POSITIVE = E4M3[:127]  # 0 .. 448, ascending


def e4m3_codes(x):
    """Nearest codes, ties to the even one; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.searchsorted(_POSITIVE, a).clip(1, 126)
    lo = hi - 1
    below, above = a - _POSITIVE[lo], _POSITIVE[hi] - a
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), pick + 128 * np.signbit(x), 127).astype(np.uint8)


def block_scale(x):
    """The least power of two s >= 2^-100 with |x| <= 448 s for the finite x."""
    x = np.abs(np.asarray(x, np.float64))
    top = float(x[np.isfinite(x)].max(initial=0.0))
    e = -100
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def block_codes(x, s):
    """Codes of a block's values at scale s, whose values float32 and bfloat16 hold: those that would
    round to 2^128 (|x| beyond 248 2^120) get the one below."""
    x = np.asarray(x, np.float64) / s
    near = np.isfinite(x) & (np.abs(x) * s >= 248.0 * 2.0 ** 120)
    return e4m3_codes(np.where(near, np.copysign(240.0, x), x))


class CacheOracle:
    """One sequence's keys or values, [tokens, heads, d], as its blocks hold them."""

    def __init__(self, heads, d):
        self.heads, self.d, self.n = heads, d, 0
        self.codes = np.zeros((0, heads, BLOCK, d), np.uint8)
        self.scale = np.zeros((0, heads))

    def append(self, x):
        x = np.asarray(x, np.float64)
        end = self.n + x.shape[0]
        blocks = -(-end // BLOCK)
        grow = blocks - self.codes.shape[0]
        self.codes = np.concatenate([self.codes, np.zeros((grow, self.heads, BLOCK, self.d), np.uint8)])
        self.scale = np.concatenate([self.scale, np.zeros((grow, self.heads))])
        for blk in range(self.n // BLOCK, blocks):
            lo, hi = max(self.n - blk * BLOCK, 0), min(end - blk * BLOCK, BLOCK)
            for h in range(self.heads):
                rows = x[blk * BLOCK + lo - self.n:blk * BLOCK + hi - self.n, h]
                if rows.shape[0] == 0:
                    continue
                s = block_scale(rows)
                if lo > 0:
                    old = self.scale[blk, h]
                    s = max(s, old)
                    self.codes[blk, h, :lo] = e4m3_codes(E4M3[self.codes[blk, h, :lo]] * old / s)
                self.codes[blk, h, lo:hi] = block_codes(rows, s)
                self.scale[blk, h] = s
        self.n = end
        return self

    def values(self):
        v = E4M3[self.codes] * self.scale[:, :, None, None]
        return v.transpose(0, 2, 1, 3).reshape(-1, self.heads, self.d)[:self.n]


def record(keys, values, blk, head):
    """The bytes of a block's record (the last 8 are unused)."""
    d = keys.d
    part = lambda o: o.codes[blk, head].reshape(BLOCK, d // 32, 32).transpose(1, 0, 2).reshape(-1)  # noqa: E731
    scales = np.array([keys.scale[blk, head], values.scale[blk, head]], np.float32)
    return np.concatenate([part(keys), part(values), scales.view(np.uint8)])
