"""Plain 64-bit reference of the 8-bit key/value cache and its attention, and
the tolerances its users take, for the GPU tests.  Shares no code with the
library."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 32
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def least_scale(amax: float) -> float:
    """2^e, e the smallest integer >= -64 with amax <= 127 * 2^e; NaN if amax is not finite."""
    if not math.isfinite(amax):
        return math.nan
    if amax == 0.0:
        return 2.0 ** -64
    e = math.frexp(amax)[1] - 8
    while amax > 127.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -64)


class Cache:
    """The cache as lists of tokens: codes [len][Hkv][D] and scales [blocks][Hkv] per sequence, keys then values."""

    def __init__(self, B, Hkv, D):
        self.Hkv, self.D = Hkv, D
        self.q = [[np.zeros((0, Hkv, D)) for _ in range(B)] for _ in range(2)]
        self.s = [[np.zeros((0, Hkv)) for _ in range(B)] for _ in range(2)]

    def write(self, b, k, v, at=None):
        """Rows k, v ([n][Hkv][D] f64) become tokens at .. of sequence b (default: appended)."""
        for i, x in enumerate((k, v)):
            q, s = self.q[i][b], self.s[i][b]
            base = len(q) if at is None else at
            end = base + len(x)
            q = np.concatenate([q[:base], np.zeros((end - base, self.Hkv, self.D))])
            nb = -(-end // BLOCK)
            s = np.concatenate([s[:-(-base // BLOCK)], np.zeros((nb - -(-base // BLOCK), self.Hkv))])
            for blk in range(base // BLOCK, nb):
                lo, hi = max(base, blk * BLOCK), min(end, blk * BLOCK + BLOCK)
                if lo >= hi:
                    continue
                kept = slice(blk * BLOCK, lo)
                for h in range(self.Hkv):
                    new = x[lo - base:hi - base, h]
                    amax = float(np.max(np.abs(new))) if np.all(np.isfinite(new)) else math.nan
                    s1 = least_scale(amax)
                    if lo > blk * BLOCK:
                        s0 = s[blk, h]
                        s1 = math.nan if math.isnan(s0) or math.isnan(s1) else max(s0, s1)
                        if not math.isnan(s1):
                            q[kept, h] = np.rint(q[kept, h] * s0 / s1)
                    s[blk, h] = s1
                    q[lo:hi, h] = 0 if math.isnan(s1) else np.rint(new / s1)
            self.q[i][b], self.s[i][b] = q, s

    def values(self, i, b, lo=0, hi=None):
        """Tokens lo .. hi - 1 as [n][Hkv][D]."""
        hi = len(self.q[i][b]) if hi is None else hi
        at = np.arange(lo, hi)
        return self.q[i][b][at] * self.s[i][b][at // BLOCK][:, :, None]


def attend(cache, b, q, scale, causal, window):
    """Rows q [n][Hq][D] f64, the last of sequence b: (o, lse, sum of weights times |v|, largest |v| seen, sum |q k|)."""
    n, Hq, D = q.shape
    k, v = cache.values(0, b), cache.values(1, b)
    L, g = len(k), Hq // cache.Hkv
    o, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    mass, top = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    reach = np.zeros((n, Hq))
    for i in range(n):
        p = L - n + i
        lo, hi = (max(0, p - window + 1) if window else 0, p + 1) if causal else (0, L)
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
            s = scale * (kk @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            z = w.sum()
            o[i, h] = w @ vv / z
            lse[i, h] = m + np.log(z)
            mass[i, h] = w @ np.abs(vv) / z
            top[i, h] = np.abs(vv).max()
            reach[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return o, lse, mass, top, reach


def bound(o, mass, top, reach, out):
    """How far an output may be from the 64-bit one.
    Weights are rounded to 11 bits (2^-11 of each term).  A score is a sum of D <= 128 products in f32: its error is at
    most D 2^-24 = 2^-17 of the sum of the products' magnitudes, and the weight moves by as much relative to itself, up
    and, through the normaliser, down: 2 * 2^-17 * reach; the exponential, the sums and the products add less than 2^-14.
    Weights below 2^-38 of the largest are dropped: 2^-20 of the largest value covers 2^18 of them.
    The output rounds once: half an ulp, which is 2^-p of the value's power of two with p = 8 (bf16), 11 (f16; 2^-25
    below its normal range) or 24 (f32) significant bits."""
    e = mass * (2.0 ** -11 + 2.0 ** -14 + (2.0 ** -16 * reach)[..., None]) + 2.0 ** -20 * top[..., None]
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
    return e + u * np.exp2(np.floor(np.log2(np.abs(o) + e + 1e-300))) + (2.0 ** -25 if out == "f16" else 0.0)


def lse_bound(lse, reach):
    """A score's error (2^-17 of the products' magnitudes), the sum's (2^-14 relative) and the f32 result's."""
    return 2.0 ** -16 * reach + 2.0 ** -14 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
