"""Plain 64-bit definitions of the MXFP4 format and its products, and of the
whole expert layer for a few tokens (numpy), the reference of their tests.
Shares no code with the HIP library."""
from __future__ import annotations

import numpy as np

from .fp8_experts import route

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MX = 32
NAN = 255


def row_scales(K):
    """Scale bytes of a row: one per 32 columns, padded to whole blocks of 128."""
    return 4 * (-(-K // 128))


def encode(q):
    """E2M1 codes of q: the nearest value, a tie to the even code, saturating."""
    a = np.minimum(np.abs(np.asarray(q, dtype=np.float64)), 6.0)
    code = np.zeros(a.shape, dtype=np.uint8)
    best = np.full(a.shape, np.inf)
    for c in list(range(0, 8, 2)) + list(range(1, 8, 2)):       # even codes first: they keep ties
        d = np.abs(a - VALUES[c])
        code = np.where(d < best, c, code).astype(np.uint8)
        best = np.minimum(d, best)
    return code | (np.signbit(q).astype(np.uint8) << 3)


def decode(code):
    return np.where(code >= 8, -1.0, 1.0) * VALUES[np.asarray(code) & 7]


def scale_value(s):
    s = np.asarray(s, dtype=np.float64)
    return np.where(s == NAN, np.nan, np.exp2(np.where(s == NAN, 0.0, s) - 127.0))


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def swiglu(x):
    K = x.shape[-1] // 2
    g, u = x[..., :K], x[..., K:]
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def quantize(v):
    """v [M, K] -> packed codes [M, K / 2], scale bytes [M, 4 * ceil(K / 128)]."""
    v = np.asarray(v, dtype=np.float64)
    M, K = v.shape
    b = v.reshape(M, -1, MX)
    bad = ~np.isfinite(b).all(2)
    amax = np.abs(np.where(bad[..., None], 0.0, b)).max(2)
    e = np.maximum(np.frexp(amax)[1] - 1 - 2, -127)
    e = np.where(amax > 0, e, -127)
    codes = encode(np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(np.float64))[..., None])
    scales = np.zeros((M, row_scales(K)), dtype=np.uint8)
    scales[:, :K // MX] = np.where(bad, NAN, e + 127)
    return pack(np.where(bad[..., None], 0, codes).astype(np.uint8).reshape(M, K)), scales


def dequantize(packed, scales):
    v = decode(unpack(packed))
    K = v.shape[-1]
    return v * np.repeat(scale_value(scales[..., :K // MX]), MX, axis=-1)


def product(a, w):
    """(a @ w^T, the sum of the terms' magnitudes) of values in 64 bits."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def fp8_block_values(values, scale):
    N, K = values.shape[-2:]
    s = np.repeat(np.repeat(np.asarray(scale, dtype=np.float64), 128, -1)[..., :K], 128, -2)[..., :N, :]
    return values * s


def int4_values(q, scale, group):
    """q [.., N, K] signed codes, scale [.., G, N]."""
    K = q.shape[-1]
    return q * np.repeat(np.swapaxes(np.asarray(scale, dtype=np.float64), -1, -2), K if group == -1 else group, -1)


def moe(x, logits, topk, w13, w2, add=None, w13_size=None, w2_size=None, **routing):
    """The layer in 64 bits on weights given as values: w13 [E, 2 I, H], w2 [E, H, I]. Returns the output and two
    magnitudes for its tolerance: how far the output moves per relative error of the first products' terms, and the sum
    of the second's terms. `w13_size`, `w2_size`: what the terms' weights count there, |w13| and |w2| if not given."""
    ids, weights = route(logits, topk, **routing)
    T, H = x.shape
    I = w2.shape[2]
    y, first, second = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(topk):
            e = ids[t, j]
            if e < 0:
                continue
            size13 = np.abs(w13[e]) if w13_size is None else w13_size[e]
            size2 = np.abs(w2[e]) if w2_size is None else w2_size[e]
            up = w13[e] @ x[t]
            upm = size13 @ np.abs(x[t])
            g, u = up[:I], up[I:]
            with np.errstate(over="ignore", invalid="ignore"):
                s = 1.0 / (1.0 + np.exp(-g))
            mid = g * s * u * weights[t, j]
            # the slope of silu is at most 1.1
            moved = np.abs(weights[t, j]) * (1.1 * upm[:I] * np.abs(u) + np.abs(g * s) * upm[I:])
            y[t] += w2[e] @ mid
            first[t] += size2 @ moved
            second[t] += size2 @ np.abs(mid)
    if add is not None:
        y = y + add
        second = second + np.abs(add)
    return y, first, second
