"""Plain 64-bit model of the 8-bit paged KV cache (include/slora.h, "KV cache
in the pool"), written from its definitions: rotation by positions, block
ranges and codes, attention over the cached values.  It keeps one array of
codes per sequence, layer and head, and shares no code with the library.
"""
from __future__ import annotations

import numpy as np

INT8, FP8 = 0, 1
HALVES, NEIGHBOURS = 0, 1
TOP = {INT8: 127.0, FP8: 448.0}


def e4m3(x):
    """Nearest e4m3 number of fp32 values (ties to even): 3 bits of fraction, exponents -6 .. 8, subnormals below."""
    x = np.asarray(x, np.float32).astype(np.float64)
    _, e = np.frexp(np.where(x == 0, 1.0, x))                    # |x| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def nearest(code, x):
    """Nearest code; only a value above its subnormal (rounded) range meets the ends."""
    return np.clip(np.rint(x), -127.0, 127.0) if code == INT8 else e4m3(np.asarray(x, np.float64).astype(np.float32))


def angles(n_positions, rot, base=10000.0):
    """fp32 table [n_positions, rot]: cosines, then sines."""
    half = rot // 2
    a = np.arange(n_positions, dtype=np.float64)[:, None] * base ** (-np.arange(half) / max(half, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate(x, cs, rot, pairs):
    """x [n, heads, dim] rotated by the rows of cs [n, rot], in 64 bits."""
    y = np.array(x, np.float64)
    if rot == 0:
        return y
    half = rot // 2
    first = np.arange(half) if pairs == HALVES else 2 * np.arange(half)
    second = first + (half if pairs == HALVES else 1)
    c, s = (np.asarray(t, np.float64)[:, None, :] for t in (cs[:, :half], cs[:, half:]))
    a, b = y[..., first], y[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def rotation_error(x, cs, rot, pairs):
    """Bound on fp32 rotation's error before its last rounding: one rounding of a product and one of the sum, 2^-24 of
    at most |a c| + |b s| each."""
    y = np.abs(rotate(np.abs(x), np.abs(cs) if rot else None, rot, pairs))
    if rot:     # |a| |c| - |b| |s| in one half: take the other sign there
        flipped = np.abs(cs).copy()
        flipped[:, rot // 2:] *= -1
        y = np.maximum(y, np.abs(rotate(np.abs(x), flipped, rot, pairs)))
    return 2.0 ** -23 * y


class KvModel:
    """Sequences of one cache: codes and ranges per (sequence, layer, what), what 0 = keys, 1 = values."""

    def __init__(self, code, n_heads, n_kv, dim, block, rot=0, pairs=HALVES, cs=None):
        self.code, self.n_heads, self.n_kv, self.dim, self.block = code, n_heads, n_kv, dim, block
        self.rot, self.pairs, self.cs = rot, pairs, cs
        self.codes, self.range = {}, {}

    def length(self, seq, layer=0):
        return self.codes[seq, layer, 0].shape[0] if (seq, layer, 0) in self.codes else 0

    def rotated(self, x, start):
        return rotate(x, self.cs[start:start + len(x)] if self.rot else None, self.rot, self.pairs)

    def append(self, seq, layer, k, v):
        start = self.length(seq, layer)
        self._store(seq, layer, 0, self.rotated(k, start))
        self._store(seq, layer, 1, np.asarray(v, np.float64))

    def _store(self, seq, layer, what, x):
        key, top, bt = (seq, layer, what), TOP[self.code], self.block
        codes = self.codes.get(key, np.zeros((0, self.n_kv, self.dim)))
        ranges = self.range.get(key, np.zeros((0, self.n_kv)))
        start, end = len(codes), len(codes) + len(x)
        codes = np.concatenate([codes, np.zeros_like(x)])
        blocks = -(-end // bt)
        ranges = np.concatenate([ranges, np.zeros((blocks - len(ranges), self.n_kv))])
        for b in range(start // bt, blocks if len(x) else 0):
            lo, hi = max(start, b * bt), min(end, (b + 1) * bt)
            for h in range(self.n_kv):
                part = x[lo - start:hi - start, h]
                with np.errstate(over="ignore", invalid="ignore"):
                    peak = np.abs(part).astype(np.float32).max()
                held = ranges[b, h]
                grown = np.float64(np.nan if not np.isfinite(peak) or np.isnan(held) else max(held, np.float64(peak)))
                if np.isnan(grown):
                    codes[b * bt:hi, h] = 0
                elif grown > 0:
                    if grown != held:
                        codes[b * bt:lo, h] = nearest(self.code, codes[b * bt:lo, h] * (held / grown))
                    codes[lo:hi, h] = nearest(self.code, part * (top / grown))
                ranges[b, h] = grown
        self.codes[key], self.range[key] = codes, ranges

    def values(self, seq, layer, what, first=0, last=None):
        """Cached values of tokens first .. last, in 64 bits."""
        codes, ranges = self.codes[seq, layer, what], self.range[seq, layer, what]
        last = len(codes) if last is None else last
        r = ranges[np.arange(first, last) // self.block][:, :, None]
        return codes[first:last] * r / TOP[self.code]

    def attend(self, seq, layer, q, start, scale, window=0, length=None):
        """Rows q [n, n_heads, dim] (rotated) at positions start, start + 1, ... over the first `length` tokens (all by
        default).  Returns the output and, per output, sum_j w_j |v_j|, the largest sum of |scale q k| over the seen
        keys and sum_j |v_j| / sum_j exp(s_j - max s) for error bounds."""
        k, v = (self.values(seq, layer, w, 0, length) for w in (0, 1))
        q = np.asarray(q, np.float64)
        n, g = len(q), self.n_heads // self.n_kv
        out, weight, reach, spread = (np.zeros((n, self.n_heads, self.dim)) for _ in range(4))
        for t in range(n):
            p = start + t
            lo = max(0, p - window + 1) if window else 0
            for h in range(self.n_heads):
                kk, vv = k[lo:p + 1, h // g], v[lo:p + 1, h // g]
                s = scale * (kk @ q[t, h])
                with np.errstate(invalid="ignore"):
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                out[t, h] = w @ vv
                weight[t, h] = w @ np.abs(vv)
                reach[t, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[t, h]))).max()
                spread[t, h] = np.abs(vv).sum(0) / e.sum()
        return out, weight, reach, spread
