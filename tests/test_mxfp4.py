"""GPU parity of the MXFP4 path against its 64-bit definitions
(oracle/mxfp4.py): quantization, its inverse, the products (dense, grouped, and
from 16-bit activations), and the path in one piece.

Tolerances are bounds of the arithmetic, u = 2^-24 the fp32 half step:
- without an activation the quantizer's scales and codes are exact;
- with one, v carries expf (2 ulp), a sum, a division and a product: 8 u
  relative, so that a code may be the other one next to a border by that much;
- products: 32 products of a block are multiples of a quarter of its scale, below
  2^13 of them: their sum is exact. Each MFMA adds two blocks' sums to the fp32
  accumulator, at most 3 roundings per 64 columns, and splits, waves and the bias
  add at most 32 more; then half a step of the output type.
"""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import fp8_experts as F
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FLOOR = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}           # half the smallest fp16 subnormal


def say(*a):
    print(*a, flush=True)


def rng_for(*a):
    return np.random.default_rng([int(v) for v in a])


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def half_step(y, dt):
    return np.abs(y) * (torch.finfo(DT[dt]).eps / 2) + FLOOR[dt]


def product_tol(y, mag, dt, K):
    return half_step(y, dt) * (1 + 1e-6) + (3 * (K // 64 + 1) + 32) * U * mag


def check(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300))))


def matrix(r, M, K, spread=3):
    """Random codes, and scales around 1 over a few binary orders; the padding holds NaN scales, which nothing may read."""
    codes = r.integers(0, 256, (M, K // 2)).astype(np.uint8)
    scales = np.full((M, O.row_scales(K)), O.NAN, dtype=np.uint8)
    scales[:, :K // 32] = r.integers(127 - spread, 128 + spread, (M, K // 32))
    return codes, scales


# ------------------------------------------------------------------ quantization

@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (2, 96), (5, 128), (1, 160), (64, 2048), (7, 2880), (129, 416), (1, 14336)])
@pytest.mark.parametrize("dt", list(DT))
def test_quantize(M, K, dt):
    r = rng_for(M, K, len(dt))
    x = gpu(r.standard_normal((M, K)) * np.exp2(r.integers(-9, 10, (M, K // 32)).repeat(32, 1)), DT[dt])
    say("quantize", M, K, dt)
    codes, scales = ops.w4_mxfp4_quantize(x)
    want = O.quantize(x.double().cpu().numpy())
    assert np.array_equal(host(scales), want[1])
    assert np.array_equal(O.decode(O.unpack(host(codes))), O.decode(O.unpack(want[0])))
    for out in DT:
        v = ops.w4_mxfp4_dequantize(codes, scales, out_dtype=DT[out])
        exact = torch.from_numpy(O.dequantize(*want)).to(DT[out])
        assert torch.equal(v.cpu(), exact), out


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_borders(dt):
    """Every border of E2M1 and its neighbours at scales over the type's whole range, subnormal ones among them; zeros of
    both signs; NaN and infinities, which take their block only."""
    fi = torch.finfo(DT[dt])
    rows = []
    lo, hi = (-24, 13) if dt == "f16" else (-133 if dt == "bf16" else -149, 125)
    for e in range(lo, hi, 1):
        s = 2.0 ** e
        v = np.array([5.0, 4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 6.0, 0.0, -0.0, -0.25, -0.75, -5.0, 7.0, 0.3]) * s
        t = torch.from_numpy(np.concatenate([v, v * (1 + fi.eps)]))
        rows.append(t.to(DT[dt]))
    x = torch.stack(rows)
    bad = torch.randn(8, 256, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).to(DT[dt])
    bad[0, 5], bad[1, 40], bad[2, 255] = float("nan"), float("inf"), -float("inf")
    bad[3] = 0.0
    bad[4] = -0.0
    bad[5] = fi.max
    bad[6] = fi.min
    for m in (x, bad):
        say("borders", dt, tuple(m.shape))
        codes, scales = ops.w4_mxfp4_quantize(m.to(DEV))
        want = O.quantize(m.double().numpy())
        assert np.array_equal(host(scales), want[1])
        assert np.array_equal(O.decode(O.unpack(host(codes))), O.decode(O.unpack(want[0])))
        v = host(ops.w4_mxfp4_dequantize(codes, scales, out_dtype=torch.float32)).astype(np.float64)
        assert np.array_equal(v, O.dequantize(*want), equal_nan=True)


@pytest.mark.parametrize("M,K", [(1, 32), (9, 224), (64, 2048)])
@pytest.mark.parametrize("dt", list(DT))
def test_quantize_swiglu(M, K, dt):
    r = rng_for(M, K, 7)
    x = gpu(r.standard_normal((M, 2 * K)) * 3, DT[dt])
    say("swiglu", M, K, dt)
    codes, scales = (host(t) for t in ops.w4_mxfp4_quantize(x, act="swiglu"))
    v = O.swiglu(x.double().cpu().numpy())
    b = np.abs(v).reshape(M, -1, 32).max(2)
    low, high = (np.frexp(b * (1 + s * 8 * U))[1] - 3 + 127 for s in (-1, 1))
    sc = scales[:, :K // 32]
    assert ((sc == low) | (sc == high)).all() and not scales[:, K // 32:].any()
    step = np.exp2(sc.astype(np.float64) - 127).repeat(32, 1)
    near = np.abs(np.minimum(np.abs(v) / step, 6.0)[..., None] - O.VALUES).min(-1) * step
    off = np.abs(np.clip(v, -6 * step, 6 * step) - O.dequantize(codes, scales))
    assert (off <= near + 16 * U * np.abs(v)).all()


def test_quantize_strided_rows_and_padding():
    x = torch.randn(37, 512, device=DEV).bfloat16()
    for view in (x[:, 64:64 + 160], x[::2, :96]):
        codes, scales = ops.w4_mxfp4_quantize(view)
        want = O.quantize(view.double().cpu().numpy())
        assert np.array_equal(host(scales), want[1])
        assert np.array_equal(O.decode(O.unpack(host(codes))), O.decode(O.unpack(want[0])))
    assert ops.w4_mxfp4_quantize(x[:0])[0].shape == (0, 256)


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(16, dtype=np.uint8)[::-1], (256, 4))   # [256, 64]
    scales = np.arange(256, dtype=np.uint8)[:, None].repeat(4, 1)
    for dt in DT:
        got = ops.w4_mxfp4_dequantize(gpu(codes), gpu(scales), out_dtype=DT[dt])
        want = torch.from_numpy(O.dequantize(codes, scales)).to(DT[dt])
        assert torch.equal(got.cpu().nan_to_num(nan=-123.0), want.nan_to_num(nan=-123.0)), dt


# ------------------------------------------------------------------ products

SHAPES = [(1, 8, 32), (1, 136, 64), (2, 264, 4096), (15, 40, 96), (16, 8200, 288), (16, 512, 2880), (17, 8, 32),
          (17, 136, 160), (33, 256, 512), (64, 264, 2880), (65, 128, 256), (100, 520, 4128), (200, 4096, 1024),
          (129, 136, 768), (257, 264, 224), (1000, 776, 544)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", list(DT))
def test_gemm(M, N, K, dt):
    r = rng_for(M, N, K)
    (a, sa), (w, sw) = matrix(r, M, K), matrix(r, N, K)
    bias = gpu(r.standard_normal(N), DT[dt]) if (M + N) % 2 else None
    say("gemm", M, N, K, dt)
    got = ops.w4_mxfp4_gemm(gpu(a), gpu(sa), gpu(w), gpu(sw), bias=bias, out_dtype=DT[dt])
    y, mag = O.product(O.dequantize(a, sa), O.dequantize(w, sw))
    if bias is not None:
        b = bias.double().cpu().numpy()
        y, mag = y + b, mag + np.abs(b)
    check(got, y, product_tol(y, mag, dt, K), (M, N, K, dt))
    again = ops.w4_mxfp4_gemm(gpu(a), gpu(sa), gpu(w), gpu(sw), bias=bias, out_dtype=DT[dt])
    assert torch.equal(got, again)


@pytest.mark.parametrize("M,N,K", [(3590, 3528, 352), (4096, 3328, 768), (200, 14344, 544), (1000, 2056, 1056),
                                   (320, 2184, 8224)])
@pytest.mark.parametrize("dt", list(DT))
def test_gemm_large_tiles(M, N, K, dt):
    """Tiles of 256 x 256 and of 128 x 128, with and without splits, ragged ones and a partial last step among them; compared
    in fp64 on the GPU."""
    r = rng_for(M, N, K)
    (a, sa), (w, sw) = matrix(r, M, K), matrix(r, N, K)
    say("gemm large", M, N, K, dt)
    got = ops.w4_mxfp4_gemm(gpu(a), gpu(sa), gpu(w), gpu(sw), out_dtype=DT[dt])
    av, wv = gpu(O.dequantize(a, sa)), gpu(O.dequantize(w, sw))
    y, mag = host(av @ wv.t()), host(av.abs() @ wv.abs().t())
    check(got, y, product_tol(y, mag, dt, K), (M, N, K, dt))


@pytest.mark.parametrize("M,N,K", [(1, 264, 4096), (16, 40, 96), (16, 8200, 288), (16, 264, 4160), (17, 136, 160), (200, 264, 2880),
                                   (300, 512, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_linear_is_quantize_and_gemm(M, N, K, dt):
    """From 16-bit activations: the same numbers as the two calls, to the bit, whatever the rows quantize to."""
    r = rng_for(M, N, K)
    x = r.standard_normal((M, K)) * np.exp2(r.integers(-12, 6, (M, K // 32)).repeat(32, 1))
    x[0, :32] = 0.0
    x = gpu(x, DT[dt])
    w, sw = (gpu(t) for t in matrix(r, N, K))
    bias = gpu(r.standard_normal(N), DT[dt]) if K % 256 else None
    say("linear", M, N, K, dt)
    got = ops.w4_mxfp4_linear(x, w, sw, bias=bias)
    a, sa = ops.w4_mxfp4_quantize(x)
    want = ops.w4_mxfp4_gemm(a, sa, w, sw, bias=bias, out_dtype=DT[dt])
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_linear_nonfinite_rows(M, dt):
    """A NaN or an infinity in a row makes that row NaN, and no other."""
    r = rng_for(M, 3)
    K, N = 320, 264
    x = r.standard_normal((M, K))
    bad = sorted({0, M // 2, M - 1})
    for i, m in enumerate(bad):
        x[m, (37 * i + 5) % K] = [np.nan, np.inf, -np.inf][i % 3]
    w, sw = (gpu(t) for t in matrix(r, N, K))
    got = host(ops.w4_mxfp4_linear(gpu(x, DT[dt]), w, sw).float())
    assert np.isnan(got[bad]).all()
    good = [m for m in range(M) if m not in bad]
    assert np.isfinite(got[good]).all()


def segments(r, E, R, kind):
    if kind == "even":
        counts = np.full(E, R // E)
    elif kind == "one":
        counts = np.zeros(E, dtype=int)
        counts[E // 2] = R
    else:
        counts = r.multinomial(R, r.dirichlet(np.ones(E) * 0.3))
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("E,R,N,K", [(1, 1, 8, 32), (8, 8, 136, 96), (64, 64, 264, 288), (4, 100, 136, 160), (8, 700, 264, 416),
                                     (3, 1000, 520, 224), (4, 5600, 2056, 288), (6, 9000, 2056, 288), (16, 2500, 4104, 288), (64, 64, 264, 4128), (3, 20, 136, 4256)])
@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_grouped(E, R, N, K, kind, dt):
    r = rng_for(E, R, N, K)
    T = max(1, R // 3)
    offsets = segments(r, E, R, kind)
    row_token = r.integers(0, T, R).astype(np.int32) if (N // 8) % 2 else None
    if row_token is None:
        T = R
    elif R > 4:
        row_token[1], row_token[R - 1] = -1, T             # rows of zeros
    (a, sa), (w, sw) = matrix(r, T, K), matrix(r, E * N, K)
    w, sw = w.reshape(E, N, -1), sw.reshape(E, N, -1)
    out = torch.full((R, N), 7.0, dtype=DT[dt], device=DEV)
    say("grouped", E, R, N, K, kind, dt, row_token is not None)
    ops.w4_mxfp4_grouped_gemm(gpu(a), gpu(sa), None if row_token is None else gpu(row_token), gpu(offsets), gpu(w), gpu(sw),
                              out=out)
    av = O.dequantize(a, sa)
    rows = np.arange(R) if row_token is None else row_token
    av = np.where(((rows >= 0) & (rows < T))[:, None], av[np.clip(rows, 0, T - 1)], 0.0)
    y, mag = np.full((R, N), 7.0), np.zeros((R, N))
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        y[s], mag[s] = O.product(av[s], O.dequantize(w[e], sw[e]))
    tol = product_tol(y, mag, dt, K)
    tol[offsets[-1]:] = 0.0                                  # rows past the last segment are left as they were
    check(out, y, tol, (E, R, N, K, kind))


def test_grouped_behind_the_last_segment():
    r = rng_for(5)
    E, R, N, K = 6, 900, 264, 128
    offsets = np.array([0, 0, 200, 203, 203, 500, 640], dtype=np.int32)
    (a, sa), (w, sw) = matrix(r, R, K), matrix(r, E * N, K)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.w4_mxfp4_grouped_gemm(gpu(a), gpu(sa), None, gpu(offsets), gpu(w.reshape(E, N, -1)), gpu(sw.reshape(E, N, -1)), out=out)
    assert (out[640:] == 7.0).all() and not (out[:640] == 7.0).all()


# ------------------------------------------------------------------ the path in one piece

@pytest.mark.parametrize("T", [1, 5, 64, 700])
def test_path(T):
    """Route, quantize, product over the experts, gate and quantize, down product, combine: each stage against the
    definition on the stage's own inputs."""
    r = rng_for(T, 11)
    E, topk, H, I = 16, 4, 416, 160
    x = gpu(r.standard_normal((T, H)), torch.bfloat16)
    logits = gpu(r.standard_normal((T, E)), torch.float32)
    w13, s13 = matrix(r, E * 2 * I, H)
    w2, s2 = matrix(r, E * H, I)
    s13, s2 = s13 - (s13 != O.NAN) * np.uint8(4), s2 - (s2 != O.NAN) * np.uint8(4)
    ids, weights, row_token, offsets, row_of = ops.w4_route(logits, topk)
    xq, xs = ops.w4_mxfp4_quantize(x)
    h = ops.w4_mxfp4_grouped_gemm(xq, xs, row_token, offsets, gpu(w13).view(E, 2 * I, -1), gpu(s13).view(E, 2 * I, -1))
    aq, asc = ops.w4_mxfp4_quantize(h, act="swiglu")
    y = ops.w4_mxfp4_grouped_gemm(aq, asc, None, offsets, gpu(w2).view(E, H, -1), gpu(s2).view(E, H, -1))
    out = ops.w4_combine(y, row_of, weights, add=x)
    off, tok = host(offsets), host(row_token)
    xv = O.dequantize(host(xq), host(xs))
    hv, av = h.double().cpu().numpy(), O.dequantize(host(aq), host(asc))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        v, mag = O.product(xv[tok[s]], O.dequantize(w13.reshape(E, 2 * I, -1)[e], s13.reshape(E, 2 * I, -1)[e]))
        check(h[s], v, product_tol(v, mag, "bf16", H), ("up", e))
        v, mag = O.product(av[s], O.dequantize(w2.reshape(E, H, -1)[e], s2.reshape(E, H, -1)[e]))
        check(y[s], v, product_tol(v, mag, "bf16", I), ("down", e))
    v, mag = F.combine(y.double().cpu().numpy(), host(row_of), host(weights), add=x.double().cpu().numpy())
    check(out, v, half_step(v, "bf16") * (1 + 1e-6) + (topk + 2) * U * mag, "combine")


def test_captured_and_on_another_stream():
    """The linear layer captured into a graph and replayed between eager calls, and calls on a stream of their own."""
    r = rng_for(2)
    K, N = 512, 264
    w, sw = (gpu(t) for t in matrix(r, N, K))
    for M in (4, 200):
        x = gpu(r.standard_normal((M, K)), torch.bfloat16)
        out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        ws = ops.w4_mxfp4_linear_workspace(M, N, K, device=DEV)
        want = ops.w4_mxfp4_linear(x, w, sw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = ops.w4_mxfp4_linear(x, w, sw, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.w4_mxfp4_linear(x, w, sw, out=out, workspace=ws)
        for k in range(4):
            x.copy_(gpu(r.standard_normal((M, K)), torch.bfloat16))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ops.w4_mxfp4_linear(x, w, sw)), (M, k)


def test_captured_products():
    """A gated quantization, a split product and a grouped one of few rows in one graph; every replay equals the eager calls
    on the same inputs, with eager calls of the same operators between them."""
    r = rng_for(5)
    M, N, K, E = 100, 544, 4128, 4
    w, sw = (gpu(t) for t in matrix(r, N, K))
    we, se = (t.view(E, N // 4, -1) for t in (w[:N // 4 * E], sw[:N // 4 * E]))
    offsets = gpu(np.array([0, 3, 3, 9, 20], dtype=np.int32))
    x = gpu(r.standard_normal((M, 2 * K)), torch.float16)
    a = (torch.empty(M, K // 2, dtype=torch.uint8, device=DEV), torch.empty(M, O.row_scales(K), dtype=torch.uint8, device=DEV))
    out = torch.empty(M, N, dtype=torch.float32, device=DEV)
    rows = torch.zeros(20, N // 4, dtype=torch.float16, device=DEV)
    ws = ops.w4_mxfp4_gemm_workspace(M, N, K, device=DEV)
    assert ws.numel() > 0

    def run(a, out, rows, ws):
        ops.w4_mxfp4_quantize(x, act="swiglu", out=a)
        ops.w4_mxfp4_gemm(*a, w, sw, out=out, workspace=ws)
        ops.w4_mxfp4_grouped_gemm(a[0][:20], a[1][:20], None, offsets, we, se, out=rows)

    say("captured products")
    graph = torch.cuda.CUDAGraph()
    run(a, out, rows, ws)
    with torch.cuda.graph(graph):
        run(a, out, rows, ws)
    for k in range(4):
        x.copy_(gpu(r.standard_normal((M, 2 * K)), torch.float16))
        out.zero_()
        rows.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = tuple(torch.empty_like(t) for t in a), torch.empty_like(out), torch.empty_like(rows), torch.empty_like(ws)
        run(*eager)
        assert torch.equal(out, eager[1]) and torch.equal(rows, eager[2]), k
        assert torch.equal(a[0], eager[0][0]) and torch.equal(a[1], eager[0][1]), k
