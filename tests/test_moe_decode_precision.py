"""w4_moe_decode keeps what lies between its two products in fp32: seen through the residual.

One column of x, one row pair of w13 and one column of w2 are alone other than zero, so both products are exact; with the
residual add = -fp16(y) the output is what fp16 leaves of y, and an error of y shows 2^11 times as large.

Tolerance, u = 2^-24, relative to |y|: expf 2 u, its sum with 1, the quotient, the product with the up row and the sum
of the parts of the second product u each: 6 u, granted as 8; add and y lie within a factor of 2, so their fp32 sum is exact;
the rest, at most 2^-11 |y|, is rounded at 2^-11 of itself, 4 u, or by fp16's half smallest step, 2^-25. A middle of 16 bits is off by up to 2^-17 = 128 u.
"""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def sparse(fmt, E, N, K, at):
    """(codes, scales) of E matrices [N, K] with the values {(e, n, k): v} and zeros elsewhere; v in -4, 2, 3, 4."""
    if fmt == "int4":
        q = np.zeros((E, N, K), dtype=np.int8)
        for i, v in at.items():
            q[i] = v
        scale = torch.ones((E, 1, N), dtype=torch.float16, device=DEV)
        return ops.w4_repack(torch.from_numpy(q).to(DEV), ops.W4_LAYOUT_I8_NK, K, N, batch=E), scale
    if fmt == "fp8_block":
        w = torch.zeros((E, N, K))
        for i, v in at.items():
            w[i] = v
        return w.to(torch.float8_e4m3fn).to(DEV), torch.ones((E, -(-N // 128), -(-K // 128)), device=DEV)
    codes = np.zeros((E, N, K), dtype=np.uint8)
    for i, v in at.items():
        codes[i] = O.encode(v)
    scales = np.full((E, N, O.row_scales(K)), 127, dtype=np.uint8)
    return torch.from_numpy(O.pack(codes)).to(DEV), torch.from_numpy(scales).to(DEV)


@pytest.mark.parametrize("T,E,H", [(1, 16, 256), (2, 16, 256), (7, 32, 256), (32, 16, 256), (7, 32, 6144), (32, 8, 6144)])
@pytest.mark.parametrize("fmt", ["fp8_block", "mxfp4", "int4"])
def test_the_middle_is_fp32(fmt, T, E, H):
    r = np.random.default_rng([T, E, H])
    I = 256
    row, column, values = r.integers(0, I, E), r.integers(0, H, E), r.choice([-4.0, 2.0, 3.0, 4.0], (E, 64))
    rows = r.permutation(H)[:64]
    w13, s13 = sparse(fmt, E, 2 * I, H, {(e, row[e] + h * I, column[e]): (2.0, 3.0)[h] for e in range(E) for h in (0, 1)})
    w2, s2 = sparse(fmt, E, H, I, {(e, n, row[e]): values[e, i] for e in range(E) for i, n in enumerate(rows)})
    for turn in range(8):
        choice = r.integers(0, E, T)
        x = np.zeros((T, H))
        x[np.arange(T), column[choice]] = r.uniform(2.0, 40.0, T) * np.where(r.random(T) < 0.25, -0.05, 1.0)
        x = torch.from_numpy(x).to(DEV, torch.float16)
        logits = torch.zeros((T, E), device=DEV)
        logits[torch.arange(T), torch.from_numpy(choice)] = 30.0
        v = x.double().cpu().numpy()[np.arange(T), column[choice]]
        middle = 2.0 * v / (1.0 + np.exp(-2.0 * v)) * 3.0 * v
        y = np.zeros((T, H))
        y[:, rows] = middle[:, None] * values[choice]
        add = torch.from_numpy(-y).to(DEV, torch.float16)
        print("middle", fmt, T, E, H, turn, flush=True)
        got = ops.w4_moe_decode(x, logits, 1, w13, s13, w2, s2, fmt=fmt, add=add).double().cpu().numpy()
        off = (np.abs(got - (y + add.double().cpu().numpy()))[:, rows] - 2.0 ** -25) / np.abs(y[:, rows])
        assert off.max() <= 12 * U, (turn, float(off.max() / U))
        rest = np.delete(got, rows, axis=1)
        assert (rest == 0).all()
