"""The list operators in numpy: AdamW with states in 32 or 8 bits, the
gradients' sum of squares, and the states' 8-bit form.

TEST INFRASTRUCTURE: see oracle/__init__.py.  Written from the formulas.
Where the library rounds every fp32 operation once, so do these (numpy's
float32 operations are IEEE, one rounding each); what the library leaves to
an accuracy is computed in float64.
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
F = np.float32


def bf16(bits):
    """bf16 bit patterns (uint16) as float32."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(F)


def to_bf16(x):
    """Nearest even; NaN to quiet NaN."""
    u = np.ascontiguousarray(x, F).view(np.uint32)
    r = (u + np.uint32(0x7fff) + ((u >> 16) & 1)) >> 16
    nan = (u & 0x7fffffff) > 0x7f800000
    return np.where(nan, (u >> 16) | 0x40, r).astype(np.uint16)


def mean(G):
    """[W][n] float32 -> the fp32 mean, summed in rank order."""
    with np.errstate(all="ignore"):
        s = G[0].copy()
        for x in G[1:]:
            s = s + x
        return s / F(len(G))


def constants(hp, t):
    """(b1, 1-b1, b2, 1-b2, lr/(1-b1^t), sqrt(1-b2^t), 1-lr*wd, eps): double,
    rounded to fp32 once."""
    lr, b1, b2, eps, wd = (float(F(x)) for x in hp)
    return tuple(F(x) for x in (b1, 1 - b1, b2, 1 - b2, lr / (1 - b1 ** t),
                                (1 - b2 ** t) ** 0.5, 1 - lr * wd, eps))


def coefficient(sumsq, max_norm):
    """The clipping coefficient, or None where the step writes nothing."""
    if not np.isfinite(sumsq) or sumsq < 0:
        return None
    norm = float(sumsq) ** 0.5
    return F(float(F(max_norm)) / norm) if norm > F(max_norm) else F(1)


def moments(g, m, v, hp, t):
    """fp32 m, v and the correctly rounded root of v."""
    b1, omb1, b2, omb2 = constants(hp, t)[:4]
    with np.errstate(all="ignore"):
        m = b1 * m + omb1 * g
        v = b2 * v + omb2 * (g * g)
        return m, v, np.sqrt(v)


def weights(w, m, root, hp, t):
    """fp32, one rounding per operation."""
    ss, bc2s, dec, eps = constants(hp, t)[4:]
    with np.errstate(all="ignore"):
        return w * dec - ss * (m / (root / bc2s + eps))


def weights64(w, m, root, hp, t):
    """(w*dec, update) from the fp32 constants, in float64."""
    ss, bc2s, dec, eps = (float(x) for x in constants(hp, t)[4:])
    w, m, root = (x.astype(np.float64) for x in (w, m, root))
    with np.errstate(all="ignore"):
        return w * dec, ss * (m / (root / bc2s + eps))


def encode(x, top):
    """(codes as int64, scales) of fp32 values, block by block.  top: 127
    (signed) or 255 (values that are not negative)."""
    x = np.asarray(x, F)
    nb = -(-len(x) // BLOCK)
    q = np.zeros(nb * BLOCK, np.int64)
    S = np.zeros(nb, F)
    with np.errstate(all="ignore"):
        for b in range(nb):
            blk = x[b * BLOCK:(b + 1) * BLOCK]
            a = np.abs(blk)
            if not np.all(np.isfinite(blk)):
                S[b] = np.nan
                continue
            A = a.max()
            if A < F(2.0 ** -100):
                continue
            S[b] = A * F(1 / top ** 2)
            y = (a * (F(top ** 2) / A)).astype(np.float64)
            # the whole number with (q - 1/2)^2 <= y < (q + 1/2)^2
            k = np.floor(np.sqrt(y)).astype(np.int64)
            k += (k + 0.5) ** 2 <= y
            if top == 255:
                k = np.maximum(k, a > 0)
            q[b * BLOCK:b * BLOCK + len(blk)] = \
                np.where(np.signbit(blk), -k, k)
    return q[:len(x)], S


FADE = 9


def faded(q, m, blank):
    """Codes q of fp32 values m, as a step holds them: where `blank` (no
    gradient on any rank) and another of the block is not, codes of up to FADE
    are rounded towards zero."""
    q, m = np.array(q), np.asarray(m, F)
    with np.errstate(all="ignore"):
        for b in range(0, len(m), BLOCK):
            s = slice(b, b + BLOCK)
            A = np.abs(m[s]).max()
            if blank[s].all() or not A >= F(2.0 ** -100):
                continue
            y = np.abs(m[s]) * (F(127 ** 2) / A)
            k = np.abs(q[s])
            q[s] -= np.sign(q[s]) * (blank[s] & (k <= FADE) & (k * k > y))
    return q


def decode(q, S):
    """fp32 values of codes."""
    q = np.asarray(q).astype(F)
    S = np.repeat(np.asarray(S, F), BLOCK)[:len(q)]
    with np.errstate(all="ignore"):
        return (q * np.abs(q)) * S


def hold(m, v):
    """(m codes, m scales, v codes, v scales) of fp32 m and v."""
    with np.errstate(all="ignore"):
        return (*encode(m, 127), *encode(np.sqrt(np.asarray(v, F)), 255))


def stands_for(mq, ms, vq, vs):
    """fp32 m and v of codes."""
    r = decode(vq, vs)
    with np.errstate(all="ignore"):
        return decode(mq, ms), r * r


def sumsq(means):
    """float64 sum of squares of fp32 means."""
    return sum(float(np.sum(np.square(g.astype(np.float64))))
               for g in means)
