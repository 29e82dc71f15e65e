"""Plain 64-bit definitions of the FP8 expert path (numpy), the reference of
its tests: routing and the row plan, E4M3 block quantization, block-scaled
FP8 products (dense and over expert segments), combine. Shares no code with
the HIP library; E4M3 encoding and decoding come from w4_oracle."""
from __future__ import annotations

import numpy as np

from .w4_oracle import e4m3_decode, e4m3_encode

BLOCK = 128
F32_MAX = float(np.finfo(np.float32).max)


def route(logits, topk, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """ids int32 and weights float64 [T, topk], one token at a time."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, topk), -1, dtype=np.int32)
    weights = np.zeros((T, topk))
    for t in range(T):
        x = np.minimum(logits[t], F32_MAX)
        open_ = x > -np.inf                                   # false for NaN too
        s = np.zeros(E)
        if open_.any():
            if score == "softmax":
                s[open_] = np.exp(x[open_] - x[open_].max())
                s /= s.sum()
            else:
                with np.errstate(over="ignore"):
                    s[open_] = 1.0 / (1.0 + np.exp(-x[open_]))
        c = s.copy()
        if bias is not None:
            c = s + np.asarray(bias, dtype=np.float64)
            open_ = open_ & (c > -np.inf)
        if n_groups > 1:
            size = E // n_groups
            values = []
            for g in range(n_groups):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if open_[e]), reverse=True)[:group_top]
                values.append(sum(best) if best else -np.inf)
            order = sorted(range(n_groups), key=lambda g: (-values[g], g))
            for g in order[topk_groups:]:
                open_[g * size:(g + 1) * size] = False
        key = x if bias is None else c
        chosen = sorted((e for e in range(E) if open_[e]), key=lambda e: (-key[e], e))[:topk]
        w = np.array([s[e] for e in chosen])
        if renorm and len(chosen):
            w = w / max(w.sum(), 1e-300)
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    return ids, weights


def plan(ids, E):
    """row_token [T * topk], expert_offsets [E + 1], row_of [T, topk] of the ids."""
    T, topk = ids.shape
    row_token = np.full(T * topk, -1, dtype=np.int32)
    row_of = np.full((T, topk), -1, dtype=np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    at = 0
    by = [[] for _ in range(E)]
    for t in range(T):
        for j in range(topk):
            if ids[t, j] >= 0:
                by[ids[t, j]].append((t, j))
    for e in range(E):
        offsets[e] = at
        for t, j in by[e]:
            row_token[at] = t
            row_of[t, j] = at
            at += 1
    offsets[E] = at
    return row_token, offsets, row_of


def silu_gate(x):
    """x [M, 2K] -> x[:, :K] * sigmoid(x[:, :K]) * x[:, K:] in float64."""
    x = np.asarray(x, dtype=np.float64)
    K = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :K] / (1.0 + np.exp(-x[:, :K])) * x[:, K:]


def block_quantize(v):
    """v [M, K] float32 -> (E4M3 codes uint8, scales float32): both divisions in correctly rounded float32."""
    v = np.asarray(v, dtype=np.float32)
    M, K = v.shape
    KB = -(-K // BLOCK)
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((M, KB), dtype=np.float32)
    for b in range(KB):
        blk = v[:, b * BLOCK:(b + 1) * BLOCK]
        s = (np.abs(blk).max(axis=1) / np.float32(448.0)).astype(np.float32)
        scales[:, b] = s
        nz = s > 0
        codes[nz, b * BLOCK:(b + 1) * BLOCK] = e4m3_encode(blk[nz] / s[nz][:, None])
    return codes, scales


def block_gemm(a, a_scale, w, w_scale, bias=None):
    """(y, magnitude) float64 [M, N]: the product and the sum of its terms' magnitudes."""
    av, wv = e4m3_decode(a).astype(np.float64), e4m3_decode(w).astype(np.float64)
    N, K = wv.shape
    y = np.zeros((av.shape[0], N))
    mag = np.zeros_like(y)
    for b in range(-(-K // BLOCK)):
        k = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        s = a_scale[:, b].astype(np.float64)[:, None] * np.repeat(w_scale[:, b].astype(np.float64), BLOCK)[None, :N]
        y += (av[:, k] @ wv[:, k].T) * s
        mag += (np.abs(av[:, k]) @ np.abs(wv[:, k]).T) * np.abs(s)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
        mag = mag + np.abs(np.asarray(bias, dtype=np.float64))
    return y, mag


def grouped_gemm(a, a_scale, row_token, offsets, w, w_scale):
    """(y, magnitude) of rows 0 .. offsets[-1]."""
    E, N = w.shape[0], w.shape[1]
    y = np.zeros((int(offsets[E]), N))
    mag = np.zeros_like(y)
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        t = r if row_token is None else row_token[r]
        if len(r):
            y[r], mag[r] = block_gemm(a[t], a_scale[t], w[e], w_scale[e])
    return y, mag


def combine(y, row_of, weights, add=None):
    """(out, magnitude) float64 [T, N]."""
    y = np.asarray(y, dtype=np.float64)
    T, topk = row_of.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(topk):
        have = (row_of[:, j] >= 0) & (row_of[:, j] < y.shape[0])
        term = weights[have, j].astype(np.float64)[:, None] * y[row_of[have, j]]
        out[have] += term
        mag[have] += np.abs(term)
    if add is not None:
        out = out + np.asarray(add, dtype=np.float64)
        mag = mag + np.abs(np.asarray(add, dtype=np.float64))
    return out, mag
