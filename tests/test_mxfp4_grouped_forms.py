"""w4_mxfp4_grouped_gemm in each of its forms (rows streamed, tiles of 64, 128, 192 and 256 rows), with gathered rows and
with rows in segment order, at 1, 3 and 9 steps of 256 columns; the larger tiles with several items per block, across experts,
empty ones among them. Against the definition in 64 bits.

Tolerance, u = 2^-24: the sum of a block of 32 products is exact, an MFMA adds two of them to the fp32 accumulator in at most
3 roundings, and 32 more are granted for the waves' sums; then half a step of the output type.
"""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
FLOOR = {"bf16": 0.0, "f16": 2.0 ** -25}


def matrix(g, *shape):
    """Random codes on the GPU, scales around 1; the padding holds NaN scales, which nothing may read."""
    *rows, K = shape
    codes = torch.randint(0, 256, (*rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.full((*rows, O.row_scales(K)), O.NAN, dtype=torch.uint8, device=DEV)
    scales[..., :K // 32] = torch.randint(124, 131, (*rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    return codes, scales


def values(codes, scales):
    grid = torch.tensor([*O.VALUES, *(-O.VALUES)], dtype=torch.float64, device=DEV)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    s = torch.exp2(scales[..., :v.shape[-1] // 32].double() - 127.0)
    return v * s.repeat_interleave(32, -1)


def segments(r, E, R, kind):
    if kind == "even":
        counts = np.full(E, R // E)
    else:
        counts = r.multinomial(R, r.dirichlet(np.ones(E)))
        counts[[0, E // 2, E - 1]] = 0                       # experts without rows; output rows behind the last segment
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# E, R, N, K
STREAMED = [(6, 40, 136, 4128), (70, 300, 264, 4352)]
TILES_64 = [(6, 170, 264, 256), (6, 170, 264, 544), (6, 170, 136, 2080)]
TILES_128 = [(5, 500, 264, 256), (5, 500, 520, 544), (5, 450, 136, 2080)]
TILES_192 = [(40, 6000, 4104, 256), (40, 6000, 4104, 544), (40, 5900, 4104, 2080)]
TILES_256 = [(6, 9000, 4104, 256), (6, 9000, 4104, 544), (6, 8900, 4104, 2080)]


@pytest.mark.parametrize("E,R,N,K", STREAMED + TILES_64 + TILES_128 + TILES_192 + TILES_256)
@pytest.mark.parametrize("kind", ["even", "ragged"])
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dt", list(DT))
def test_forms(E, R, N, K, kind, gathered, dt):
    r = np.random.default_rng([E, R, N, K])
    g = torch.Generator(DEV).manual_seed(R + K)
    T = max(1, R // 3) if gathered else R
    off = segments(r, E, R, kind)
    tok = r.integers(0, T, R).astype(np.int32) if gathered else None
    if gathered:
        tok[1], tok[R // 2] = -1, T                          # rows of zeros
    a, sa = matrix(g, T, K)
    w, sw = matrix(g, E, N, K)
    out = torch.full((R, N), 7.0, dtype=DT[dt], device=DEV)
    token = torch.from_numpy(tok).to(DEV) if gathered else None
    offsets = torch.from_numpy(off).to(DEV)
    print("grouped form", E, R, N, K, kind, gathered, dt, flush=True)
    ops.w4_mxfp4_grouped_gemm(a, sa, token, offsets, w, sw, out=out)
    av = values(a, sa)
    if gathered:
        t = token.long()
        av = torch.where(((t >= 0) & (t < T))[:, None], av[t.clamp(0, T - 1)], 0.0)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start == s.stop:
            continue
        wv = values(w[e], sw[e]).t().contiguous()
        y, size = av[s] @ wv, av[s].abs() @ wv.abs()
        tol = y.abs() * (torch.finfo(DT[dt]).eps / 2 * (1 + 1e-6)) + FLOOR[dt] + (3 * (K // 64 + 1) + 32) * U * size
        bad = ~((out[s].double() - y).abs() <= tol)
        assert not bad.any(), (e, int(bad.sum()))
    assert (out[int(off[-1]):] == 7.0).all()                 # rows behind the last segment stay as they were
    again = torch.full_like(out, 7.0)
    ops.w4_mxfp4_grouped_gemm(a, sa, token, offsets, w, sw, out=again)
    assert torch.equal(out, again)
