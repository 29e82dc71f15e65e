"""GPU parity of the whole expert layer for a few tokens (w4_moe_decode) against
its 64-bit definition (oracle/mxfp4.py), in each weight format.

Tolerance, u = 2^-24 the fp32 half step: the operands are exact, so the first
products carry at most one rounding per term and a few for scales and splits,
(H + 64) u of their terms, passed on through the gate and the second product; the
gate's own arithmetic 16 u; the middle is held as two bf16 numbers, each the
nearest: 2^-18; the second products' terms (topk I + 64) u; then half a step of
the output type. int4 products are formed as x (u) - 8 x with codes u of 0..15, so
their terms count 23 steps of the scale.
"""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import mxfp4 as O
from oracle.w4_oracle import e4m3_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FLOOR = {"bf16": 0.0, "f16": 2.0 ** -25}
FMTS = ["fp8_block", "mxfp4", "int4"]


def say(*a):
    print(*a, flush=True)


def rng_for(*a):
    return np.random.default_rng([int(v) for v in a])


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def matrix(fmt, r, E, N, K, group=128):
    """(what the call takes, values, sizes of the terms' weights) of E random matrices [N, K]."""
    if fmt == "fp8_block":
        codes = r.integers(0, 256, (E, N, K)).astype(np.uint8)
        codes[(codes & 0x7F) > 0x70] = 0x30                  # not the largest, and no NaN
        scale = (r.random((E, -(-N // 128), -(-K // 128))) * 0.01 + 0.002).astype(np.float32)
        values = O.fp8_block_values(e4m3_decode(codes).astype(np.float64), scale)
        return (gpu(codes), gpu(scale)), values, np.abs(values)
    if fmt == "mxfp4":
        codes = r.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
        scale = np.full((E, N, O.row_scales(K)), O.NAN, dtype=np.uint8)          # the padding is NaN
        scale[..., :K // 32] = r.integers(118, 124, (E, N, K // 32))
        values = O.dequantize(codes, scale)
        return (gpu(codes), gpu(scale)), values, np.abs(values)
    q = r.integers(-8, 8, (E, N, K)).astype(np.int8)
    G = 1 if group == -1 else K // group
    scale = (r.random((E, G, N)) * 0.02 + 0.002).astype(np.float16)
    tiled = ops.w4_repack(gpu(q), ops.W4_LAYOUT_I8_NK, K, N, batch=E)
    return (tiled, gpu(scale)), O.int4_values(q, scale, group), O.int4_values(np.full_like(q, 23), scale, group)


def layer(fmt, r, E, H, I, group=128):
    return matrix(fmt, r, E, 2 * I, H, group), matrix(fmt, r, E, H, I, group)


def call(x, logits, topk, w, fmt, **kw):
    (w13, s13), (w2, s2) = w[0][0], w[1][0]
    return ops.w4_moe_decode(x, logits, topk, w13, s13, w2, s2, fmt=fmt, **kw)


def check(got, x, logits, topk, w, dt, add=None, bias=None, **routing):
    (_, w13, size13), (_, w2, size2) = w
    H, I = w2.shape[1:]
    y, first, second = O.moe(x.double().cpu().numpy(), logits.double().cpu().numpy(), topk, w13, w2,
                             add=None if add is None else add.double().cpu().numpy(), w13_size=size13, w2_size=size2,
                             bias=None if bias is None else bias.cpu().numpy(), **routing)
    tol = np.abs(y) * (torch.finfo(DT[dt]).eps / 2) * (1 + 1e-6) + FLOOR[dt]
    tol += (H + 64) * U * first + (2.0 ** -18 + 16 * U + (topk * I + 64) * U) * second
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - y) / tol)))
    return y


@pytest.mark.parametrize("T", [1, 2, 3, 8, 16, 17, 32])
@pytest.mark.parametrize("E,topk,H,I,kw", [
    (8, 2, 256, 128, {}), (4, 4, 160, 96, dict(score="sigmoid", renorm=False)), (1, 1, 32, 32, {}),
    (40, 6, 416, 224, dict(bias=True, scale=2.5)),
    (64, 8, 384, 128, dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2, bias=True, scale=2.5)),
    (300, 5, 128, 128, dict(n_groups=3, topk_groups=2, group_top=1)),
])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_layer(T, E, topk, H, I, kw, fmt, dt):
    if fmt == "int4":
        H, I = -(-H // 128) * 128, -(-I // 128) * 128
    kw = dict(kw)
    r = rng_for(T, E, topk, H, I)
    w = layer(fmt, r, E, H, I, group=-1 if E == 40 else 128)
    x = gpu(r.standard_normal((T, H)), DT[dt])
    logits = gpu(r.standard_normal((T, E)) * 2, DT[("f32", "bf16", "f16")[(T + E) % 3]])
    if T > 2:
        logits[T // 2] = -torch.inf                        # a padding token
    add = gpu(r.standard_normal((T, H)), DT[dt]) if T % 2 else None
    bias = gpu((r.standard_normal(E) * 0.1).astype(np.float32)) if kw.pop("bias", False) else None
    say("layer", T, E, topk, H, I, kw, fmt, dt)
    got = call(x, logits, topk, w, fmt, add=add, bias=bias, **kw)
    check(got, x, logits, topk, w, dt, add=add, bias=bias, **kw)
    assert torch.equal(got, call(x, logits, topk, w, fmt, add=add, bias=bias, **kw))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,topk", [(2, 64, 64), (32, 4, 1), (32, 64, 64), (9, 1024, 3)])
def test_layer_ends_of_the_routing(fmt, T, E, topk):
    """Every expert chosen by every token, all tokens at one expert, ties, and the most experts."""
    r = rng_for(T, E, topk, 5)
    H, I = 128, 128
    w = layer(fmt, r, E, H, I)
    x = gpu(r.standard_normal((T, H)), torch.bfloat16)
    logits = gpu(r.integers(-2, 3, (T, E)), torch.float32)
    if topk == 1:
        logits[:, 2] = 9.0
    say("ends", fmt, T, E, topk)
    check(call(x, logits, topk, w, fmt), x, logits, topk, w, "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,I,topk,T", [(2048, 1408, 4, 1), (7168, 256, 2, 5), (256, 2048, 8, 20), (6272, 128, 8, 32),
                                        (7168, 128, 3, 17)])
def test_layer_long_sums(fmt, H, I, topk, T):
    r = rng_for(H, I)
    w = layer(fmt, r, 8, H, I)
    x = gpu(r.standard_normal((T, H)), torch.float16)
    logits = gpu(r.standard_normal((T, 8)), torch.float32)
    say("long", fmt, H, I, topk, T)
    check(call(x, logits, topk, w, fmt), x, logits, topk, w, "f16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 2])
def test_blocks_that_take_several_column_tiles(fmt, T):
    """More tiles than blocks that route for themselves."""
    r = rng_for(T, 31)
    E, topk, H, I = 64, 24 * (3 - T), 128, 768 // T
    w = layer(fmt, r, E, H, I)
    x = gpu(r.standard_normal((T, H)), torch.bfloat16)
    logits = gpu(r.standard_normal((T, E)), torch.float32)
    say("several tiles", fmt, T)
    check(call(x, logits, topk, w, fmt), x, logits, topk, w, "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [2, 20])
def test_no_expert_and_values_that_are_not_finite(fmt, dt, T):
    """Tokens without an expert get the residual or zero; NaN and infinities stay in their token's row; a NaN in the
    weights of an expert reaches the tokens that chose it alone."""
    r = rng_for(T, 77)
    E, topk, H, I = 8, 2, 256, 128
    w = layer(fmt, r, E, H, I)
    x = gpu(r.standard_normal((T, H)), DT[dt])
    logits = torch.full((T, E), -torch.inf, device=DEV)
    say("none", fmt, dt, T)
    assert (call(x, logits, topk, w, fmt) == 0).all()
    add = gpu(r.standard_normal((T, H)), DT[dt])
    assert torch.equal(call(x, logits, topk, w, fmt, add=add), add)
    logits = gpu(r.standard_normal((T, E)), torch.float32)
    logits[0, :] = -torch.inf
    logits[0, :2] = 1.0                                     # token 0: experts 0 and 1; the others: not these
    logits[1:, :2] = -torch.inf
    good = call(x, logits, topk, w, fmt)
    bad_x = x.clone()
    bad_x[0, 3], bad_x[0, 200] = torch.nan, torch.inf
    got = call(bad_x, logits, topk, w, fmt)
    assert got[0].isnan().all() and torch.equal(got[1:], good[1:])
    for which in (0, 1):                                    # w13, then w2
        t, s = (v.clone() for v in w[which][0])
        if fmt == "mxfp4":
            s[0] = O.NAN
        elif fmt == "fp8_block":
            t[0] = 0x7F
        else:
            s[0] = torch.nan
        broken = [((t, s),) if i == which else w[i] for i in (0, 1)]
        got = call(x, logits, topk, broken, fmt)
        assert got[0].isnan().all() and torch.equal(got[1:], good[1:]), which


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_mxfp4_scales_over_their_range(dt):
    """Weights far above and below 1, beyond fp16: the scales go into the operands as bf16."""
    r = rng_for(9)
    E, topk, H, I, T = 4, 2, 128, 64, 3
    w = []
    for N, K, centre in ((2 * I, H, 127 - 40), (H, I, 127 + 70)):
        codes = r.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
        scale = np.full((E, N, O.row_scales(K)), O.NAN, dtype=np.uint8)
        scale[..., :K // 32] = r.integers(centre - 3, centre + 4, (E, N, K // 32))
        v = O.dequantize(codes, scale)
        w.append(((gpu(codes), gpu(scale)), v, np.abs(v)))
    x = gpu(r.standard_normal((T, H)), DT[dt])
    logits = gpu(r.standard_normal((T, E)), torch.float32)
    say("scales", dt)
    check(call(x, logits, topk, w, "mxfp4"), x, logits, topk, w, dt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 12])
def test_captured_strided_in_place_and_on_another_stream(fmt, T):
    r = rng_for(T, 3)
    E, topk, H, I = 16, 4, 256, 128
    w = layer(fmt, r, E, H, I)
    x = gpu(r.standard_normal((T, H)), torch.bfloat16)
    wide = gpu(r.standard_normal((T, 2 * E)), torch.float32)
    logits = wide[:, E:]
    say("captured", fmt, T)
    want = call(x, logits.contiguous(), topk, w, fmt, add=x)
    assert torch.equal(call(x, logits, topk, w, fmt, add=x), want)
    out = x.clone()
    assert torch.equal(call(x, logits, topk, w, fmt, add=out, out=out), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(x, logits, topk, w, fmt, add=x, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = ops.w4_moe_decode_workspace(T, E, topk, H, I, device=DEV)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, logits, topk, w, fmt, out=out, workspace=ws)
    for k in range(4):
        x.copy_(gpu(r.standard_normal((T, H)), torch.bfloat16))
        wide.copy_(gpu(r.standard_normal((T, 2 * E)), torch.float32))
        out.zero_()
        ws.fill_(0xFF)                                      # nothing in it has to survive
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(x, logits, topk, w, fmt)), k


@pytest.mark.parametrize("fmt", FMTS)
def test_two_calls_at_once(fmt):
    """On streams and workspaces of their own: what each gives alone."""
    r = rng_for(41)
    E, topk, H, I = 16, 4, 512, 256
    w = layer(fmt, r, E, H, I)
    sets = [(gpu(r.standard_normal((T, H)), torch.bfloat16), gpu(r.standard_normal((T, E)), torch.float32)) for T in (2, 9, 32)]
    say("at once", fmt)
    want = [call(x, lg, topk, w, fmt) for x, lg in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[call(x, lg, topk, w, fmt, stream=s) for _ in range(8)] for (x, lg), s in zip(sets, streams)]
    torch.cuda.synchronize()
    for v, several in zip(want, got):
        assert all(torch.equal(v, g) for g in several)


def test_tensors_of_another_device(monkeypatch):
    """Calls with tensors or a stream of another device than the current one are refused."""
    r = rng_for(43)
    w, x = layer("mxfp4", r, 4, 64, 32), gpu(r.standard_normal((2, 64)), torch.bfloat16)
    logits = gpu(r.standard_normal((2, 4)), torch.float32)
    offsets = gpu(np.array([0, 1, 1, 2, 2], dtype=np.int32))
    a, sa = ops.w4_mxfp4_quantize(x)
    (w13, s13), side = w[0][0], torch.cuda.Stream()
    calls = [lambda **kw: ops.w4_mxfp4_quantize(x, **kw), lambda **kw: ops.w4_mxfp4_dequantize(a, sa, **kw),
             lambda **kw: ops.w4_mxfp4_gemm(a, sa, w13[0], s13[0], **kw),
             lambda **kw: ops.w4_mxfp4_linear(x, w13[0], s13[0], **kw),
             lambda **kw: ops.w4_mxfp4_grouped_gemm(a, sa, None, offsets, w13, s13, **kw),
             lambda **kw: call(x, logits, 2, w, "mxfp4", **kw)]
    for f in calls:
        f()
        f(stream=side)
    torch.cuda.synchronize()
    monkeypatch.setattr(ops, "_current_device", lambda: 1)
    for f in calls:
        with pytest.raises(ValueError, match="current device is cuda:1"):
            f()
        with pytest.raises(ValueError, match="current device is cuda:1"):
            f(stream=side)


def test_nothing_to_do():
    (w13, s13), (w2, s2) = (m[0] for m in layer("mxfp4", rng_for(1), 4, 64, 32))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert ops.w4_moe_decode(x, torch.empty((0, 4), device=DEV), 2, w13, s13, w2, s2, fmt="mxfp4").shape == (0, 64)
