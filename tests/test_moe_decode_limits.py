"""w4_moe_decode at the sizes that fill LDS (32 tokens of 1024 experts, up to 64 chosen, in each form of the down
products; the plan of 1024 experts in 64 groups), and int4 weights in groups of more than 128. Against the definition in
64 bits, computed expert by expert on the GPU.

Tolerance, u = 2^-24: one rounding per term of the first products and a few for scales and splits, (H + 64) u of their terms;
16 u for the gate; (topk I + 64) u of the second products' terms; half a step of the output type. int4 products are formed
from codes of 0 to 15 and -8 times the row's sum, so their terms count 23 steps of the scale.
"""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import mxfp4 as O
from oracle.fp8_experts import route

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


class Matrices:
    """E random matrices [N, K] of a format: what the call takes, and one expert's values and the weights of its terms."""

    def __init__(self, fmt, g, E, N, K, group=128):
        def ints(low, high, *shape, dtype=torch.uint8):
            return torch.randint(low, high, shape, dtype=dtype, device=DEV, generator=g)
        self.fmt, self.K, self.group = fmt, K, K if group == -1 else group
        if fmt == "fp8_block":
            self.w = ints(0, 0x60, E, N, K) | ints(0, 2, E, N, K) << 7
            self.s = torch.rand((E, -(-N // 128), -(-K // 128)), device=DEV, generator=g) * 0.01 + 0.002
        elif fmt == "mxfp4":
            self.w = ints(0, 256, E, N, K // 2)
            self.s = torch.full((E, N, O.row_scales(K)), O.NAN, dtype=torch.uint8, device=DEV)
            self.s[..., :K // 32] = ints(118, 124, E, N, K // 32)
        else:
            self.q = ints(-8, 8, E, N, K, dtype=torch.int8)
            self.w = ops.w4_repack(self.q, ops.W4_LAYOUT_I8_NK, K, N, batch=E)
            self.s = (torch.rand((E, K // self.group, N), device=DEV, generator=g) * 0.02 + 0.002).half()

    def values(self, e):
        s = self.s[e].double()
        if self.fmt == "fp8_block":
            w = self.w[e].view(torch.float8_e4m3fn).double()
            v = w * s.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :self.K]
            return v, v.abs()
        if self.fmt == "mxfp4":
            grid = torch.tensor([*O.VALUES, *(-O.VALUES)], dtype=torch.float64, device=DEV)
            c = self.w[e]
            v = grid[torch.stack([c & 15, c >> 4], -1).flatten(-2).long()]
            v = v * torch.exp2(s[:, :self.K // 32] - 127.0).repeat_interleave(32, 1)
            return v, v.abs()
        step = s.t().repeat_interleave(self.group, 1)
        return self.q[e].double() * step, 23.0 * step


def check(fmt, T, E, topk, H, I, seed, group=128, dt=torch.bfloat16, **routing):
    g = torch.Generator(DEV).manual_seed(seed)
    w13, w2 = Matrices(fmt, g, E, 2 * I, H, group), Matrices(fmt, g, E, H, I, group)
    x = torch.randn((T, H), device=DEV, generator=g).to(dt)
    logits = torch.randn((T, E), device=DEV, generator=g)
    bias = torch.randn(E, device=DEV, generator=g) * 0.1 if routing.pop("bias", False) else None
    print("limits", fmt, T, E, topk, H, I, group, routing, flush=True)
    got = ops.w4_moe_decode(x, logits, topk, w13.w, w13.s, w2.w, w2.s, fmt=fmt, bias=bias, **routing)
    ids, weights = route(logits.double().cpu().numpy(), topk, bias=None if bias is None else bias.cpu().numpy(), **routing)
    y, first, second = (torch.zeros((T, H), dtype=torch.float64, device=DEV) for _ in range(3))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        share = torch.from_numpy(np.asarray(weights)[t, j]).to(DEV, torch.float64)[:, None]
        rows = torch.from_numpy(t).to(DEV)
        (v, size), (v2, size2) = w13.values(e), w2.values(e)
        up, upm = x[rows].double() @ v.t().contiguous(), x[rows].double().abs() @ size.t().contiguous()
        gate, u = up[:, :I], up[:, I:]
        silu = gate * torch.sigmoid(gate)
        mid = silu * u * share
        moved = share.abs() * (1.1 * upm[:, :I] * u.abs() + silu.abs() * upm[:, I:])      # silu's slope is at most 1.1
        y[rows] += mid @ v2.t().contiguous()
        first[rows] += moved @ size2.t().contiguous()
        second[rows] += mid.abs() @ size2.t().contiguous()
    tol = y.abs() * (torch.finfo(dt).eps / 2 * (1 + 1e-6)) + (2.0 ** -25 if dt == torch.float16 else 0.0)
    tol += (H + 64) * U * first + (16 + topk * I + 64) * U * second
    off = (got.double() - y).abs()
    assert (off <= tol).all(), (int((off > tol).sum()), float((off / tol).max()))
    assert torch.equal(got, ops.w4_moe_decode(x, logits, topk, w13.w, w13.s, w2.w, w2.s, fmt=fmt, bias=bias, **routing))


FMTS = ["fp8_block", "mxfp4", "int4"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [256, 6144])
@pytest.mark.parametrize("topk", [63, 64])                   # the down products' tiles of 4 rows, and of 5
def test_the_most_of_everything(fmt, H, topk):
    check(fmt, 32, 1024, topk, H, 128 if fmt == "int4" else 32, 7)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,topk,kw", [(32, 8, dict(topk_groups=16, group_top=2)), (3, 64, dict(topk_groups=64)),
                                       (2, 8, dict(topk_groups=16, group_top=2))])
def test_the_most_experts_in_groups(fmt, T, topk, kw):
    check(fmt, T, 1024, topk, 128, 128, 9, score="sigmoid", n_groups=64, bias=True, scale=2.5, **kw)


@pytest.mark.parametrize("T", [1, 5, 32])
@pytest.mark.parametrize("H,I,group", [(512, 256, 256), (1024, 512, 256), (768, 384, 384), (2048, 1024, 512), (640, 640, 640),
                                       (384, 640, -1)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_int4_groups_of_more_than_128(T, H, I, group, dt):
    check("int4", T, 8, 3, H, I, T + H, group=group, dt=dt)
