"""Attention over kv8ref's cache in 64 bits, with bounds per output type that
hold for values and scores of any size."""
from __future__ import annotations

import numpy as np

import kv8ref


def attend(cache, b, q, scale, causal, window, out):
    """(o, lse, bound of o, bound of lse) of rows q [n][Hq][D], the last of sequence b, in 64 bits.

    The bound, relative to the sum of the weighted values' magnitudes unless said otherwise.  A score: exact products,
    eight truncated sums and two roundings of at most 2^-23 of the products' magnitudes (`reach`), less than 2^-19 of it,
    once in the weight and once in the normaliser: 2^-18 reach.  The block's exponent, up to 128 in size, joins it and
    the maximum comes off: two roundings of at most 2^-18 each, as often: 2^-16.  f32 outputs: weights in two terms
    2^-22, exponential 2^-21, truncated sums 5e-6: with the exponent's less than 2^-15.  16-bit outputs: weights in one
    term 2^-11, all else 2^-14.
    Weights are fp16 numbers against a largest (weight times block scale) of at least 2^10: each is off by up to 2^-25,
    and meets codes up to 127: tokens * 2^-28 of that largest.  The output rounds once."""
    n, Hq, D = q.shape
    k, v, L = cache.values(0, b), cache.values(1, b), len(cache.q[0][b])
    vs = cache.s[1][b][np.arange(L) // kv8ref.BLOCK]
    g, o, lse, e = Hq // cache.Hkv, np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    reach = np.zeros((n, Hq))
    for i in range(n):
        p = L - n + i
        lo, hi = (max(0, p - window + 1) if window else 0, p + 1) if causal else (0, L)
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
            s = scale * (kk @ q[i, h])
            w = np.exp(s - s.max())
            z = w.sum()
            w /= z
            o[i, h], lse[i, h] = w @ vv, s.max() + np.log(z)
            reach[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            rel = (2.0 ** -15 if out == "f32" else 2.0 ** -11 + 2.0 ** -14) + 2.0 ** -18 * reach[i, h]
            e[i, h] = rel * (w @ np.abs(vv)) + (hi - lo) * 2.0 ** -28 * (w * vs[lo:hi, h // g]).max()
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
    e = e + u * np.exp2(np.floor(np.log2(np.abs(o) + e + 1e-300))) + (2.0 ** -25 if out == "f16" else 0.0)
    return o, lse, e, kv8ref.lse_bound(lse, reach)
