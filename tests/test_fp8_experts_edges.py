"""GPU tests of the FP8 expert path's edges: infinities and NaN on their way
through the quantizer and the products, sizes past one launch's threads, and
the router's plan in the int4 experts' product, routing by one wave per token,
and the precision of the products' sums."""
import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from int4_weight_quantized_amd import workloads as W
from oracle import fp8_experts as O
from oracle.w4_oracle import bf16_bits_to_f32, e4m3_decode, grouped_fp8_reference, quantize_act_fp8
from test_fp8_experts import DEV, DT, U, check, check_route, fp8_inputs, gpu, half_step, rng_for, say
from test_gpu_parity import assert_close, to_f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ infinities in the quantizer

INF, NAN = float("inf"), float("nan")
# row -> {column: value of v}; columns of the second and third 128-block
ODD = {1: {130: INF}, 2: {131: -INF}, 3: {256: INF, 257: -INF}, 4: {c: INF for c in range(128, 256)},
       5: {140: -INF, 141: NAN}, 6: {300: NAN}}


def odd_rows(dt, act):
    """x whose v has the infinities and NaN of ODD and is finite elsewhere, [8, 384] (or gate | up side by side)."""
    r = rng_for(len(dt), len(act), 31)
    v = r.standard_normal((8, 384))
    if act == "none":
        for row, at in ODD.items():
            for c, val in at.items():
                v[row, c] = val
        return gpu(v, DT[dt])
    up = 1.0 + r.random((8, 384))
    for row, at in ODD.items():
        for i, (c, val) in enumerate(at.items()):
            # +-inf by the gate, by the other factor, and (bf16) by a product past fp32's range
            if np.isnan(val):
                v[row, c] = NAN
            elif i % 2 == 0:
                v[row, c], up[row, c] = INF, np.copysign(1.5, val)
            elif dt == "bf16":
                v[row, c], up[row, c] = 2e38, np.copysign(2e38, val)
            else:
                v[row, c], up[row, c] = 2.0, val
    return gpu(np.concatenate([v, up], axis=1), DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_block_quantize_infinities(dt, act):
    """An infinity makes its block's scale +inf, its own code NaN and the finite columns' codes 0 (inf / inf and
    v / inf); a NaN in the block makes the scale NaN and every code 0. Other blocks know nothing of it."""
    say("quant infinities", dt, act)
    x = odd_rows(dt, act)
    codes, scales = ops.w4_fp8_block_quantize(x, act=act)
    d = codes.view(torch.float8_e4m3fn).float().cpu().numpy().reshape(8, 3, 128)
    s = scales.cpu().numpy()
    hit = np.zeros((8, 3), dtype=bool)
    for row, at in ODD.items():
        b = next(iter(at)) // 128
        hit[row, b] = True
        vals = np.zeros(128)
        for c, val in at.items():
            vals[c - 128 * b] = val
        if np.isnan(vals).any():
            assert np.isnan(s[row, b]) and (d[row, b] == 0).all(), row
        else:
            assert np.isposinf(s[row, b]), row
            assert np.array_equal(np.isnan(d[row, b]), np.isinf(vals)), row
            assert (d[row, b][np.isfinite(vals)] == 0).all(), row
    assert np.isfinite(s[~hit]).all() and (s[~hit] > 0).all() and np.isfinite(d[~hit]).all()
    assert (np.abs(d[~hit]).max(1) == 448).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("copies", [1, 5, 25])
def test_infinities_reach_their_rows(dt, act, copies):
    """Rows with an infinity or a NaN come out of the products as NaN whatever its sign, the others finite: streamed
    (8 rows), 64-row tiles (40), 128-row tiles (200), and over expert segments."""
    say("infinities through the product", dt, act, copies)
    x = odd_rows(dt, act).repeat(copies, 1)
    M, N, K = 8 * copies, 72, 384
    codes, scales = ops.w4_fp8_block_quantize(x, act=act)
    r = rng_for(N, K, 5)
    w = gpu(fp8_inputs(r, (3, N, K), 3))
    ws = gpu(r.uniform(1e-3, 3e-3, (3, 1, 3)).astype(np.float32))
    want = torch.tensor([row in ODD for row in range(8)], device=DEV).repeat(copies)[:, None].expand(M, N)
    for out_dt in (torch.bfloat16, torch.float16, torch.float32):
        y = ops.w4_fp8_block_gemm(codes, scales, w[0], ws[0], out_dtype=out_dt)
        assert torch.equal(torch.isnan(y), want) and torch.isfinite(y[~want]).all(), out_dt
    off = gpu(np.array([0, M // 2, M // 2, M], dtype=np.int32))
    y = ops.w4_fp8_block_grouped_gemm(codes, scales, None, off, w, ws)
    assert torch.equal(torch.isnan(y), want) and torch.isfinite(y[~want]).all()
    order = torch.arange(M - 1, -1, -1, dtype=torch.int32, device=DEV)
    y = ops.w4_fp8_block_grouped_gemm(codes, scales, order, off, w, ws, out_dtype=torch.float16)
    assert torch.equal(torch.isnan(y), want.flip(0)) and torch.isfinite(y[~want.flip(0)]).all()


# ------------------------------------------------------------------ sizes past one launch's threads (2^32)

def test_combine_past_one_launch():
    """T * N / 8 just above 2^32 (64 GiB of output): every token gets its row, none of the ranges is left out."""
    N, R = 8192, 3
    T = (1 << 32) // (N // 8) + 7
    say("combine past one launch", T, N)
    y = torch.arange(1, R * N + 1, device=DEV).remainder_(251).reshape(R, N).bfloat16()
    table = torch.cat([torch.zeros((1, N), dtype=y.dtype, device=DEV), y])
    row = (torch.arange(T, device=DEV) * 2654435761 >> 7).remainder_(4).to(torch.int32) - 1
    out = torch.full((T, N), 7.0, dtype=y.dtype, device=DEV)
    ops.w4_combine(y, row[:, None].contiguous(), torch.ones((T, 1), device=DEV), out=out)
    for t0 in range(0, T, 1 << 18):
        part = slice(t0, min(T, t0 + (1 << 18)))
        assert torch.equal(out[part], table[row[part].long() + 1]), t0


def test_block_quantize_past_one_launch():
    """More than 2^28 blocks, one per row: a pattern of 64 rows, its codes and scales repeated to the end."""
    K, P = 8, 64
    M = (1 << 28) + 3 * P + 5
    say("quant past one launch", M, K)
    g = torch.Generator(DEV).manual_seed(12)
    rows = torch.randn((P, K), device=DEV, generator=g).bfloat16()
    x = rows.repeat(M // P + 1, 1)[:M]
    codes = torch.full((M, K), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((M, 1), 7.0, device=DEV)
    ops.w4_fp8_block_quantize(x, out=(codes, scales))
    c, s = O.block_quantize(rows.float().cpu().numpy())
    c, s = gpu(e4m3_decode(c)), gpu(s)
    for m0 in range(0, M, 1 << 24):                              # a multiple of P
        part = slice(m0, min(M, m0 + (1 << 24)))
        n = part.stop - m0
        assert torch.equal(scales[part], s.repeat(n // P + 1, 1)[:n]), m0
        assert torch.equal(codes[part].view(torch.float8_e4m3fn).float(), c.float().repeat(n // P + 1, 1)[:n]), m0


def test_route_most_tokens():
    """The largest T: the choice, and the plan as a permutation ordered by expert, then token."""
    T = (1 << 28) - 64
    say("route most tokens", T)
    x = torch.empty((T, 2), dtype=torch.bfloat16, device=DEV)
    second = (torch.arange(T, device=DEV) * 40503 >> 9).remainder_(3) == 0
    x[:, 0] = 0
    x[:, 1] = torch.where(second, 1.0, -1.0)
    ids, weights, row_token, off, row_of = ops.w4_route(x, 1)
    ids, row_of = ids.view(-1), row_of.view(-1)
    assert torch.equal(ids == 1, second) and int(ids.min()) == 0 and bool((weights == 1).all())
    n0 = T - int(second.sum())
    assert off.tolist() == [0, n0, T]
    tokens = torch.arange(T, dtype=torch.int32, device=DEV)
    assert torch.equal(row_token[:n0], tokens[~second]) and torch.equal(row_token[n0:], tokens[second])
    assert torch.equal(row_token[row_of.long()], tokens)


# ------------------------------------------------------------------ the plan and the int4 experts

@pytest.mark.parametrize("E,K,N,group,T,topk", [(8, 256, 136, 128, 300, 3), (5, 512, 72, 256, 7, 2), (3, 128, 64, 128, 1, 2)])
def test_route_feeds_int4_experts(E, K, N, group, T, topk):
    """route -> quantize per token -> w4a8_grouped_gemm -> combine, with tokens that have no expert, or fewer than
    topk: their plan ends before R, the product leaves the rows past its end as they are, and combine reads none."""
    say("int4 experts", E, K, N, group, T, topk)
    d = W.moe_inputs(E, K, N, group, T, topk, seed=E + T)
    x = torch.from_numpy(d["x"].view(np.int16)).view(torch.bfloat16).to(DEV)
    r = rng_for(E, K, T)
    logits = r.standard_normal((T, E)).astype(np.float32)
    logits[T // 2] = -np.inf
    logits[T // 3, 1:] = -np.inf
    ids, weights, row_token, off, row_of = ops.w4_route(gpu(logits), topk, score="sigmoid")
    n, R = int(off[-1]), T * topk
    assert n < R and int(row_token[n:].max()) == -1
    a8, s, gs = ops.w4a8_quantize_act(x, "fp8", group)
    wt = ops.w4_repack(torch.from_numpy(d["w"]).to(DEV), ops.W4_LAYOUT_CT_NK, K, N, batch=E)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.w4a8_grouped_gemm(a8, s, gs, row_token, off, wt, gpu(d["scales"]), group, N, out=out)
    torch.cuda.synchronize()
    assert (out[n:] == 7).all()
    want_ids, _ = O.route(logits, topk, score="sigmoid")
    plan = O.plan(want_ids, E)
    rc, rs = quantize_act_fp8(bf16_bits_to_f32(d["x"]))
    assert_close(to_f64(out[:n]), grouped_fp8_reference(rc, rs, *plan[:2], d["w"], d["scales"], group), "int4 experts")
    y = ops.w4_combine(out, row_of, weights)
    want, mag = O.combine(out.double().cpu().numpy(), plan[2], weights.cpu().numpy())
    check(y, want, half_step(want, "bf16") * (1 + 1e-6) + (topk + 2) * U * mag, "combine")
    assert not y[T // 2].any()


# ------------------------------------------------------------------ routing by one wave per token

# more than 256 experts, or groups that do not fall on whole lanes of 16
WAVE = [(384, 8, {}), (512, 10, dict(renorm=False)), (512, 64, dict(score="sigmoid", scale=2.5)), (1024, 64, {}),
        (1000, 7, dict(score="sigmoid", renorm=False)), (300, 6, dict(bias=True)), (512, 5, dict(bias=True, score="sigmoid")),
        (1024, 9, dict(bias=True)), (72, 5, dict(n_groups=3, topk_groups=2, group_top=2)),
        (60, 4, dict(n_groups=4, topk_groups=2, group_top=1, bias=True, score="sigmoid")),
        (300, 5, dict(n_groups=3, topk_groups=2, group_top=2, bias=True)),
        (1024, 8, dict(n_groups=64, topk_groups=7, group_top=2, score="sigmoid")),
        (1024, 64, dict(n_groups=2, topk_groups=2, group_top=1, bias=True))]


@pytest.mark.parametrize("E,topk,kw", WAVE)
@pytest.mark.parametrize("T", [1, 63, 130])
def test_route_wave(E, topk, kw, T):
    kw = dict(kw)
    r = rng_for(T, E, topk, 8)
    x = r.standard_normal((T, E)) * 2
    bias = (r.standard_normal(E) * 0.1).astype(np.float32) if kw.pop("bias", False) else None
    check_route(gpu(x, DT[("f32", "bf16", "f16")[(T + E) % 3]]), topk, bias=bias, **kw)


# 16 lanes per token, for the same masks
LANES = [(64, 5, dict(score="sigmoid", bias=True)), (40, 6, dict(n_groups=5, topk_groups=3, group_top=2, bias=True)),
         (256, 8, dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2, bias=True, scale=2.5)), (16, 16, {})]


@pytest.mark.parametrize("E,topk,kw", WAVE + LANES)
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_route_masks_ties_and_bias_ends(E, topk, kw, dt):
    """Ties everywhere, closed experts, rows with less than topk open, the type's ends, NaN, equal groups; a bias that
    closes experts, ties others and is infinite."""
    kw = dict(kw)
    r = rng_for(E, topk, len(dt))
    T = 130
    x = r.integers(-3, 4, (T, E)).astype(np.float64)
    x[r.random((T, E)) < 0.3] = -np.inf
    x[3] = -np.inf
    x[4] = np.nan
    x[5] = torch.finfo(DT[dt]).min
    x[6, 1:] = -np.inf
    x[7, :4] = np.inf
    x[8] = np.where(np.arange(E) % 2, np.nan, 1.0)
    x[9] = torch.finfo(DT[dt]).min
    x[9, E // 2] = torch.finfo(DT[dt]).max
    x[10, :E - 2] = -np.inf                                      # the last group alone, and short
    x[64:128] = 1.0
    bias = None
    if kw.pop("bias", False):
        bias = (r.integers(-2, 3, E) * 0.125).astype(np.float32)
        bias[2], bias[5], bias[E - 3] = -np.inf, np.nan, np.inf
    check_route(gpu(x, DT[dt]), topk, bias=bias, **kw)


# ------------------------------------------------------------------ the precision of the products' sums

def small_ints(shape, g):
    """E4M3 codes of whole numbers from -8 to 16."""
    return torch.randint(-8, 17, shape, device=DEV, generator=g).float().to(torch.float8_e4m3fn)


def halves(shape, g, unit):
    """Scales of 1/2 and 1 units (a power of two)."""
    return torch.randint(1, 3, shape, device=DEV, generator=g).float() * (unit / 2)


def exact_product(a, sa, w, sw):
    """The product in float64, where it is exact."""
    K, N = a.shape[1], w.shape[0]
    a = a.float() * sa.repeat_interleave(128, 1)[:, :K]
    w = w.float() * sw.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return a.double() @ w.double().t()


def assert_rounded(got, y):
    """The output is the exact value, rounded once: every partial sum is a multiple of a quarter unit below 2^24 of them."""
    assert torch.equal(y, y.float().double())
    bad = got != y.float().to(got.dtype)
    assert not bad.any(), (int(bad.sum()), bad.numel())


PRODUCTS = [(1, 4104, 4096), (12, 8200, 2064), (40, 520, 4112), (64, 2056, 528), (200, 512, 14336), (700, 1032, 528),
            (2305, 6152, 1152)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_block_gemm_exact(M, N, K, dt):
    """Whole numbers and scales of powers of two: no sum on the way may round, in whatever order or unit it is formed
    (streamed, 64-, 128- and 256-row tiles, K splits), so each output is off by its own rounding alone."""
    say("gemm exact", M, N, K, dt)
    g = torch.Generator(DEV).manual_seed(M + N + K)
    KB, NB = -(-K // 128), -(-N // 128)
    unit = 2.0 ** -8 if dt == "f16" else 1.0                     # within fp16's range
    a, w = small_ints((M, K), g), small_ints((N, K), g)
    sa, sw = halves((M, KB), g, 1.0), halves((NB, KB), g, unit)
    bias = torch.randint(-16, 17, (N,), device=DEV, generator=g).float() * unit
    got = ops.w4_fp8_block_gemm(a, sa, w, sw, bias=bias.to(DT[dt]), out_dtype=DT[dt])
    assert_rounded(got, exact_product(a, sa, w, sw) + bias.double())


COUNTS = [[1, 0, 3, 16, 4, 2, 0, 6], [40, 0, 129, 1, 300], [700, 513, 0, 256, 31, 1100, 1, 120]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_grouped_gemm_exact(counts, gather, dt):
    """The same over segments: streamed, and tiles of 128 and 256 rows."""
    say("grouped exact", counts, gather, dt)
    E, R, N, K = len(counts), sum(counts), 3720, 1168
    g = torch.Generator(DEV).manual_seed(R)
    T = 77 if gather else R
    KB, NB = -(-K // 128), -(-N // 128)
    a, w = small_ints((T, K), g), small_ints((E, N, K), g)
    sa, sw = halves((T, KB), g, 1.0), halves((E, NB, KB), g, 2.0 ** -8 if dt == "f16" else 1.0)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rt = torch.randint(0, T, (R,), device=DEV, generator=g, dtype=torch.int32) if gather else None
    got = ops.w4_fp8_block_grouped_gemm(a, sa, rt, gpu(off), w, sw, out_dtype=DT[dt])
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        pick = rt[rows].long() if gather else rows
        assert_rounded(got[rows], exact_product(a[pick], sa[pick], w[e], sw[e]))


def normal_codes(shape, g):
    return (torch.randn(shape, device=DEV, generator=g) * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)


def assert_close_sums(got, y):
    """fp16 outputs of normal data: beside the output's own rounding, the sums are off by no more than 2e-5 (rms, of the
    result's rms), where the matrix unit's grid costs about 1e-5."""
    rms = y.pow(2).mean()
    own = (y.to(torch.float16).double() - y).pow(2).mean() / rms
    err = (got.double() - y).pow(2).mean() / rms
    assert err - own <= 2e-5 ** 2, (err.sqrt().item(), own.sqrt().item())


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_block_gemm_normal_data(M, N, K):
    g = torch.Generator(DEV).manual_seed(M + N + K)
    a, w = normal_codes((M, K), g), normal_codes((N, K), g)
    sa = torch.rand((M, -(-K // 128)), device=DEV, generator=g) * 0.006 + 0.003
    sw = torch.rand((-(-N // 128), -(-K // 128)), device=DEV, generator=g) * 2e-4 + 1e-4
    got = ops.w4_fp8_block_gemm(a, sa, w, sw, out_dtype=torch.float16)
    assert_close_sums(got, exact_product(a, sa, w, sw))
    again = ops.w4_fp8_block_gemm(a, sa, w, sw, out=torch.full_like(got, 7.0))
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))   # no order left to timing


@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_gemm_normal_data(counts):
    E, R, N, K = len(counts), sum(counts), 3720, 1168
    g = torch.Generator(DEV).manual_seed(R + 1)
    KB, NB = -(-K // 128), -(-N // 128)
    a, w = normal_codes((R, K), g), normal_codes((E, N, K), g)
    sa = torch.rand((R, KB), device=DEV, generator=g) * 0.006 + 0.003
    sw = torch.rand((E, NB, KB), device=DEV, generator=g) * 2e-4 + 1e-4
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    got = ops.w4_fp8_block_grouped_gemm(a, sa, None, gpu(off), w, sw, out_dtype=torch.float16)
    y = torch.cat([exact_product(a[off[e]:off[e + 1]], sa[off[e]:off[e + 1]], w[e], sw[e]) for e in range(E)])
    assert_close_sums(got, y)
    again = ops.w4_fp8_block_grouped_gemm(a, sa, None, gpu(off), w, sw, out=torch.full_like(got, 7.0))
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))
