"""Plain 64-bit references of a drafting step: rotary positions, attention with a mask over
kv8ref's cache, and the check of drafted tokens; and the tolerances their users take.
Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

import kv8ref


def rotate(x, pos, freq, layout, mag=1.0):
    """x [T][H][D] f64 at positions pos: channels i, i + rot/2 ("half") or 2i, 2i + 1 ("pairs")."""
    y, r = x.copy(), len(freq)
    for t, p in enumerate(pos):
        for i, f in enumerate(freq):
            # p * f reduced by whole turns first (both are exact numbers: a product of 31 and 24 bits, in 64-bit floats)
            c, s = mag * math.cos(float(p) * float(f)), mag * math.sin(float(p) * float(f))
            a, b = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
            u, v = x[t, :, a], x[t, :, b]
            y[t, :, a], y[t, :, b] = u * c - v * s, v * c + u * s
    return y


def rotate_bound(x, pos, freq, layout, mag=1.0):
    """How far a rotated channel may be off before its last rounding.  An angle is exact to 2^-33 of a turn, cosine and sine
    are off by 2^-24 (the last rounding's 2^-25, and as much for everything before it), times mag 2^-24 more, a product
    2^-24, the sum 2^-24 of itself: together below 2^-22 of |a mag| + |b mag|; 2^-30 more for the 64-bit angle of this
    reference at positions of 2^31 (2^31 f 2^-53)."""
    y, r = np.zeros_like(x), len(freq)
    for i in range(r):
        a, b = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
        far = max(abs(int(p)) for p in pos) * abs(float(freq[i])) * 2.0 ** -52
        both = (np.abs(x[:, :, a]) + np.abs(x[:, :, b])) * abs(mag) * (2.0 ** -22 + far)
        y[:, :, a] = y[:, :, b] = both
    return y


def rounding(y, out):
    """Half a step of the type at values up to y in size."""
    u, least = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 2.0 ** -150)}[out]
    return u * np.exp2(np.floor(np.log2(np.abs(y) + 1e-300))) + least


def tree(rng, n, chain=0.4):
    """Parents of n nodes, the first the root."""
    return [-1] + [i - 1 if rng.random() < chain else int(rng.integers(max(0, i - 6), i)) for i in range(1, n)]


def bits_of(parents):
    """Each node's ancestors and itself."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def words(bits, width):
    """Bit sets as int32 words [rows][width]."""
    w = np.array([[b >> 32 * i & 0xFFFFFFFF for i in range(width)] for b in bits], dtype=np.uint64).reshape(len(bits), width)
    return w.astype(np.uint32).view(np.int32)


def attend(cache, b, q, scale, bits, out):
    """(o, lse, bound of o, bound of lse) of rows q [n][Hq][D], the last of sequence b, which see all tokens before them and
    those of their bits among them.  The bounds are those of kv8tight (they count tokens, however they are chosen)."""
    n, Hq, D = q.shape
    k, v, L = cache.values(0, b), cache.values(1, b), len(cache.q[0][b])
    vs = cache.s[1][b][np.arange(L) // kv8ref.BLOCK]
    g, o, lse, e = Hq // cache.Hkv, np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    reach = np.zeros((n, Hq))
    for i in range(n):
        see = [t for t in range(L) if t < L - n or bits[i] >> (t - (L - n)) & 1]
        if not see:
            continue
        for h in range(Hq):
            kk, vv = k[see, h // g], v[see, h // g]
            s = scale * (kk @ q[i, h])
            w = np.exp(s - s.max())
            z = w.sum()
            w /= z
            o[i, h], lse[i, h] = w @ vv, s.max() + np.log(z)
            reach[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            rel = (2.0 ** -15 if out == "f32" else 2.0 ** -11 + 2.0 ** -14) + 2.0 ** -18 * reach[i, h]
            e[i, h] = rel * (w @ np.abs(vv)) + len(see) * 2.0 ** -28 * (w * vs[see, h // g]).max()
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
    e = e + u * np.exp2(np.floor(np.log2(np.abs(o) + e + 1e-300))) + (2.0 ** -25 if out == "f16" else 0.0)
    return o, lse, e, kv8ref.lse_bound(lse, reach)


def verify(P, Q, tokens, parents, u, u_last):
    """(tokens that stand and the drawn one, places of the rows that stand) of one sequence; P, Q [n][V] f64."""
    good = lambda x: np.where(x > 0, x, 0.0)
    cur, out, path = 0, [], [0]
    while True:
        p, q = good(P[cur]), None if Q is None else good(Q[cur])
        w, m, go = p.copy(), 1.0, None
        for c in range(cur + 1, len(parents)):
            if parents[c] != cur:
                continue
            x = tokens[c]
            r = 0.0 if u[c] < 0 else u[c]
            if r * (1.0 if Q is None else q[x]) * max(m, 0.0) < w[x]:
                assert w[x] > 0
                go = c
                break
            if Q is None:
                m -= w[x]
                w[x] = 0.0
            else:
                w = np.maximum(w - m * q, 0.0)
                m = w.sum()
        if go is None:
            break
        out.append(int(tokens[go]))
        path.append(go)
        cur = go
    if not w.sum() > 0:
        w = p
    if not w.sum() > 0:
        return out + [-1], path
    cum = np.cumsum(w)
    hit = np.nonzero((cum > u_last * cum[-1]) & (w > 0))[0]
    return out + [int(hit[0]) if len(hit) else int(np.nonzero(w > 0)[0][-1])], path
