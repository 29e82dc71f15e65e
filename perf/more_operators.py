"""What is measured of the MXFP4 path (4-bit floating point elements, one power
of two per 32 of them) and of the whole expert layer for a few tokens:
quantization, the products (dense and over expert segments) from 16-bit
activations, and the layer from router logits to the experts' weighted sum.

`listed()` names the fixed cases, `draw(rng)` gives more of the same ranges,
`prepare(case, seed)` makes a case's inputs on the GPU, `run(state)` makes one
pass (the plain torch form, or this library's entry points where `own` is
true), `work(case)` counts what a pass has to move and compute, and
`exact(case, seed)` gives the outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
MX = 32                         # elements per scale of the MXFP4 format
BLOCK = 128                     # the FP8 weights' scale block, along K and along N; the int4 weights' group
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
HUGE = torch.finfo(torch.float32).max
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
PLAIN_ROUTING = dict(score="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # quantization there and back (codes and scales, then the values they stand for): a few fp32 weight rows;
        # the down projection's prefill activations
        dict(name="quant_few", op="quant", M=64, K=2048, dtype="f32"),
        dict(name="quant_rows", op="quant", M=8192, K=14336, dtype="f16"),
        # the linear layer: one decode token; a ragged batch of decode tokens through the down projection with fp32
        # results; a prefill up projection
        dict(name="gemm_one", op="gemm", M=1, N=14336, K=4096, dtype="bf16", bias=False),
        dict(name="gemm_batch", op="gemm", M=200, N=4096, K=14336, dtype="f32", bias=True),
        dict(name="gemm_prefill", op="gemm", M=4096, N=14336, K=4096, dtype="bf16", bias=False),
        # experts' products: eight decode tokens (most experts hold one row or none); the gated down projection of 1024
        # tokens; a prefill batch of 65,536 routed rows, the largest case
        dict(name="experts_few", op="experts", T=8, E=64, topk=8, N=2048, K=7168, dtype="bf16", gated=False, skew=0.0),
        dict(name="experts_down", op="experts", T=1024, E=64, topk=8, N=7168, K=2048, dtype="f16", gated=True, skew=0.0),
        dict(name="experts_many", op="experts", T=8192, E=64, topk=8, N=2048, K=7168, dtype="bf16", gated=False,
             skew=0.0),
        # the whole layer: one decode token with FP8 weights; two with int4 weights and the residual added; eight with
        # MXFP4 weights and grouped sigmoid routing; a batch of 32 with a few padding tokens
        dict(name="moe_one", op="moe", T=1, E=64, topk=8, H=7168, I=2048, dtype="bf16", fmt="fp8_block", add=False,
             pad=0.0, logits="f32", **PLAIN_ROUTING),
        dict(name="moe_two_int4", op="moe", T=2, E=64, topk=8, H=7168, I=2048, dtype="bf16", fmt="int4", add=True,
             pad=0.0, logits="bf16", **PLAIN_ROUTING),
        dict(name="moe_eight_mxfp4", op="moe", T=8, E=64, topk=8, H=7168, I=2048, dtype="bf16", fmt="mxfp4", add=False,
             pad=0.0, logits="f32", score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5),
        dict(name="moe_batch", op="moe", T=32, E=64, topk=8, H=7168, I=2048, dtype="f16", fmt="fp8_block", add=False,
             pad=0.1, logits="f16", **PLAIN_ROUTING),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "experts", "moe", "moe"])
    if op == "quant":
        K = MX * _log(rng, 1, 448)
        return dict(op=op, M=_log(rng, 1, min(65536, 117440512 // K)), K=K, dtype=rng.choice(list(DTYPES)))
    if op == "gemm":
        N, K = 8 * _log(rng, 16, 1792), MX * _log(rng, 2, 448)
        M = _log(rng, 1, min(8192, max(1, 480_000_000_000 // (2 * N * K))))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(list(DTYPES)), bias=rng.random() < 0.5)
    if op == "experts":
        E = rng.choice([4, 8, 16, 32, 64, 128])
        N = 8 * _log(rng, 16, 896)
        K = MX * _log(rng, 2, min(224, max(4, 900_000_000 // (E * N * MX))))
        topk = rng.randint(1, min(8, E // 2))
        T = _log(rng, 1, min(8192, max(2, 1_800_000_000_000 // (2 * topk * N * K))))
        return dict(op=op, T=T, E=E, topk=topk, N=N, K=K, dtype=rng.choice(["bf16", "f16"]), gated=rng.random() < 0.4,
                    skew=rng.choice([0.0, 0.0, 2.0]))
    fmt = rng.choice(["fp8_block", "mxfp4", "int4"])
    unit = BLOCK if fmt == "int4" else MX
    E = rng.choice([4, 8, 16, 40, 64, 128, 256])
    H = unit * _log(rng, 2, 7168 // unit)
    I = unit * _log(rng, 1, min(2048 // unit, max(2, 900_000_000 // (3 * E * H * unit))))
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
    chosen = 1 if groups == 1 else rng.randint(1, groups)
    return dict(op=op, T=rng.choice([1, 1, 2, rng.randint(3, 16), rng.randint(9, 32)]), E=E,
                topk=rng.randint(1, min(10, chosen * (E // groups))), H=H, I=I, dtype=rng.choice(["bf16", "f16"]),
                fmt=fmt, add=rng.random() < 0.4, pad=rng.choice([0.0, 0.1]), logits=rng.choice(list(DTYPES)),
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.4, groups=groups, topk_groups=chosen,
                group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))


def _weight_bytes(fmt, n, k):
    """Bytes of an [n, k] weight matrix with its scales."""
    if fmt == "fp8_block":
        return n * k + 4 * ceil_div(n, BLOCK) * ceil_div(k, BLOCK)
    return n * k / 2 + (n * ceil_div(k, MX) if fmt == "mxfp4" else 2 * n * ceil_div(k, BLOCK))


def work(case):
    c = case
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        return {"bytes": n * SIZE[c["dtype"]] + n / 2 + n / MX + 2 * n, "flops": 3 * n}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + _weight_bytes("mxfp4", N, K) + (M + bool(c["bias"])) * N * SIZE[c["dtype"]],
                "flops": 2 * M * N * K}
    if c["op"] == "experts":
        rows, N, K = c["T"] * c["topk"], c["N"], c["K"]
        hit = c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"])     # experts that hold a row, on average
        read = 2 * (2 * rows * K if c["gated"] else c["T"] * K)
        return {"bytes": read + hit * _weight_bytes("mxfp4", N, K) + rows * N * 2, "flops": 2 * rows * N * K}
    T, H, I = c["T"], c["H"], c["I"]
    real = T * (1.0 - c["pad"])
    hit = c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** real)
    return {"bytes": hit * (_weight_bytes(c["fmt"], 2 * I, H) + _weight_bytes(c["fmt"], H, I)) +
            T * H * 2 * (3 if c["add"] else 2) + T * c["E"] * SIZE[c["logits"]],
            "flops": 2 * real * c["topk"] * 3 * H * I}


# ------------------------------------------------------------------ MXFP4 in elementary operations

def _mx_scale_values(scales):
    return scales.view(torch.float8_e8m0fnu).float()


def _mx_quantize(v):
    """fp32 [..., K] -> the elements' E2M1 values and the scale bytes, one per 32 along K."""
    b = v.reshape(*v.shape[:-1], -1, MX)
    amax = b.abs().amax(-1)
    # floor(log2 amax) - 2, biased by 127
    scale = torch.where(amax > 0, (torch.frexp(amax)[1] + (127 - 3)).clamp(min=0), 0)
    q = b * ((254 - scale) << 23).to(torch.int32).view(torch.float32)[..., None]      # times 2^(127 - scale), exactly
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), q)
    return q.view(v.shape), scale.to(torch.uint8)


def _mx_pack(q):
    """E2M1 values -> two codes per byte, the lower index in the low nibble."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    code = code.view(*q.shape[:-1], -1, 2)
    return code[..., 0] | code[..., 1] << 4


_pairs = {}


def _mx_unpack(codes):
    """Packed codes [..., K / 2] -> E2M1 values fp32 [..., K]."""
    if "e2m1" not in _pairs:
        one = torch.tensor(E2M1 + [-x for x in E2M1], device=DEV)
        _pairs["e2m1"] = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    return _pairs["e2m1"].index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], 2 * codes.shape[-1])


def _int4_unpack(codes):
    """Signed int4, two per byte, low nibble first -> fp32."""
    both = torch.stack([codes << 4 >> 4, codes >> 4], -1)
    return both.view(*codes.shape[:-1], 2 * codes.shape[-1]).float()


def _pad_scales(s):
    """Rows of scale bytes padded to whole blocks of 128 elements."""
    return torch.nn.functional.pad(s, (0, -s.shape[-1] % 4)).contiguous()


def _mx_values(codes, scales):
    q = _mx_unpack(codes)
    s = _mx_scale_values(scales[..., :q.shape[-1] // MX].contiguous())
    return (q.view(*s.shape, MX) * s[..., None]).view(q.shape)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed))


def _uniform(shape, lo, hi, g):
    return torch.rand(shape, device=DEV, generator=g) * (hi - lo) + lo


def _mx_weights(lead, N, K, g):
    """Normal weights in MXFP4: codes [*lead, N, K / 2], scales [*lead, N, padded]."""
    parts = [_mx_quantize(torch.randn((N, K), device=DEV, generator=g) * 0.02) for _ in range(math.prod(lead))]
    codes = torch.stack([_mx_pack(q) for q, _ in parts]).view(*lead, N, K // 2)
    return codes, torch.stack([_pad_scales(s) for _, s in parts]).view(*lead, N, -1)


def _weights(fmt, E, N, K, g):
    if fmt == "mxfp4":
        return _mx_weights((E,), N, K, g)
    if fmt == "fp8_block":
        w = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(E):
            w[e] = (torch.randn((N, K), device=DEV, generator=g) * 110).clamp_(-448, 448).to(w.dtype)
        return w, _uniform((E, ceil_div(N, BLOCK), ceil_div(K, BLOCK)), 1e-4, 3e-4, g)
    w = torch.empty((E, N, K // 2), dtype=torch.int8, device=DEV)
    for e in range(E):
        q = (torch.randn((N, K), device=DEV, generator=g) * 2.5).round_().clamp_(-8, 7).to(torch.int8)
        w[e] = (q[:, ::2] & 15) | q[:, 1::2] << 4
    return w, _uniform((E, K // BLOCK, N), 0.004, 0.012, g).half()


def _routing(T, E, topk, skew, g):
    """Rows (token, slot) of distinct random experts (later ones more often where skewed), ordered by expert, then token."""
    keys = torch.randn((T, E), device=DEV, generator=g) + skew * torch.linspace(0, 1, E, device=DEV)
    flat = keys.topk(topk, dim=1).indices.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return (order // topk).to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    dt = DTYPES[c["dtype"]]
    half = torch.bfloat16 if c["dtype"] == "f32" else dt                # the activations' type
    if c["op"] == "quant":
        s["x"] = torch.randn((c["M"], c["K"]), device=DEV, generator=g).to(dt)
        s["out"] = (torch.empty((c["M"], c["K"] // 2), dtype=torch.uint8, device=DEV),
                    torch.empty((c["M"], 4 * ceil_div(c["K"], BLOCK)), dtype=torch.uint8, device=DEV),
                    torch.empty((c["M"], c["K"]), dtype=torch.bfloat16, device=DEV))
    elif c["op"] == "gemm":
        s["x"] = torch.randn((c["M"], c["K"]), device=DEV, generator=g).to(half)
        s["w"], s["w_scale"] = _mx_weights((), c["N"], c["K"], g)
        s["bias"] = torch.randn(c["N"], device=DEV, generator=g).to(dt) if c["bias"] else None
        s["out"] = torch.empty((c["M"], c["N"]), dtype=dt, device=DEV)
    elif c["op"] == "experts":
        rows = c["T"] * c["topk"]
        s["row_token"], s["offsets"] = _routing(c["T"], c["E"], c["topk"], c["skew"], g)
        if c["gated"]:                                                  # the up product's rows, gate and up side by side
            s["row_token"] = None
            s["x"] = (torch.randn((rows, 2 * c["K"]), device=DEV, generator=g) * 1.5).to(dt)
        else:
            s["x"] = torch.randn((c["T"], c["K"]), device=DEV, generator=g).to(dt)
        s["w"], s["w_scale"] = _mx_weights((c["E"],), c["N"], c["K"], g)
        s["out"] = torch.empty((rows, c["N"]), dtype=dt, device=DEV)
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        x = torch.randn((T, E), device=DEV, generator=g) * 1.5
        if c["pad"]:
            x[torch.rand(T, device=DEV, generator=g) < c["pad"]] = -math.inf    # padding tokens: every expert masked
        s["logits"] = x.to(DTYPES[c["logits"]])
        s["bias"] = torch.randn(E, device=DEV, generator=g) * 0.05 if c["bias"] else None
        s["x"] = torch.randn((T, H), device=DEV, generator=g).to(dt)
        s["add"] = torch.randn((T, H), device=DEV, generator=g).to(dt) if c["add"] else None
        s["w13"], s["w13_scale"] = _weights(c["fmt"], E, 2 * I, H, g)
        s["w2"], s["w2_scale"] = _weights(c["fmt"], E, H, I, g)
        s["out"] = torch.empty((T, H), dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    from int4_weight_quantized_amd import ops
    if c["op"] == "quant":
        codes, scales, values = s["out"]
        ops.w4_mxfp4_quantize(s["x"], out=(codes, scales))
        return ops.w4_mxfp4_dequantize(codes, scales, out=values), scales.view(torch.float8_e8m0fnu)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        if c["dtype"] != "f32":
            if "ws" not in s:
                s["ws"] = ops.w4_mxfp4_linear_workspace(M, N, K, device=DEV)
            return ops.w4_mxfp4_linear(s["x"], s["w"], s["w_scale"], bias=s["bias"], out=s["out"], workspace=s["ws"])
        if "ws" not in s:
            s["ws"] = ops.w4_mxfp4_gemm_workspace(M, N, K, device=DEV)
        a, a_scale = ops.w4_mxfp4_quantize(s["x"])
        return ops.w4_mxfp4_gemm(a, a_scale, s["w"], s["w_scale"], bias=s["bias"], out=s["out"], workspace=s["ws"])
    if c["op"] == "experts":
        a, a_scale = ops.w4_mxfp4_quantize(s["x"], act="swiglu" if c["gated"] else "none")
        return ops.w4_mxfp4_grouped_gemm(a, a_scale, s["row_token"], s["offsets"], s["w"], s["w_scale"], out=s["out"])
    if "ws" not in s:
        s["ws"] = ops.w4_moe_decode_workspace(c["T"], c["E"], c["topk"], c["H"], c["I"], device=DEV)
        s["laid"] = s["w13"], s["w2"]
        if c["fmt"] == "int4":                       # the int4 kernels' tiles, laid out at load time
            s["laid"] = (ops.w4_repack(s["w13"], ops.W4_LAYOUT_S4_NK, c["H"], 2 * c["I"], batch=c["E"]),
                         ops.w4_repack(s["w2"], ops.W4_LAYOUT_S4_NK, c["I"], c["H"], batch=c["E"]))
    return ops.w4_moe_decode(s["x"], s["logits"], c["topk"], s["laid"][0], s["w13_scale"], s["laid"][1], s["w2_scale"],
                             fmt=c["fmt"], score=c["score"], bias=s["bias"], n_groups=c["groups"],
                             topk_groups=c["topk_groups"], group_top=c["group_top"], renorm=c["renorm"],
                             scale=c["scale"], add=s["add"], out=s["out"], workspace=s["ws"])


def _first(keys, k):
    """Indices of the k largest along the last dimension, the lowest index first among equals."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :k]


def _route_plain(s, c):
    """ids [T, topk] (-1: none) and weights fp32; the choice in 64 bits: it is between near values."""
    x = s["logits"].double()
    open_ = x > -math.inf                        # neither -inf nor NaN
    x = torch.where(open_, x.clamp(max=HUGE), -math.inf)
    if c["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = torch.where(open_, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    low = -math.inf
    choice = torch.where(open_, p if s["bias"] is None else p + s["bias"].double(), low)
    key = x if s["bias"] is None else choice
    if c["groups"] > 1:
        G = c["groups"]
        best = torch.sort(choice.view(-1, G, c["E"] // G), dim=2, descending=True).values[..., :c["group_top"]]
        some = best[..., 0] > low
        rank = torch.where(some, torch.where(best > low, best, 0.0).sum(2), low)
        kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, _first(rank, c["topk_groups"]), True)
        key = torch.where(kept.repeat_interleave(c["E"] // G, dim=1), key, low)
    ids = _first(key, c["topk"])
    none = torch.gather(key, 1, ids) == low
    w = torch.where(none, 0.0, torch.gather(p, 1, ids))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(none, -1, ids), (w * c["scale"]).float()


def _values(fmt, w, scale):
    """Weight matrices of the chosen experts in fp32."""
    if fmt == "mxfp4":
        return _mx_values(w, scale)
    if fmt == "fp8_block":
        N, K = w.shape[-2:]
        scale = scale.repeat_interleave(BLOCK, dim=-1)[..., :K].repeat_interleave(BLOCK, dim=-2)[..., :N, :]
        return w.float() * scale
    w = _int4_unpack(w)
    return w * scale.float().transpose(1, 2).repeat_interleave(BLOCK, dim=2)


def _run_plain(s, c):
    dt = DTYPES[c["dtype"]]
    if c["op"] == "quant":
        q, scale = _mx_quantize(s["x"].float())
        values = (q.view(c["M"], -1, MX) * _mx_scale_values(scale)[..., None]).view(q.shape)
        return values.to(torch.bfloat16), _pad_scales(scale).view(torch.float8_e8m0fnu)
    if c["op"] in ("gemm", "experts"):
        x = s["x"].float()
        if c["op"] == "experts" and c["gated"]:
            x = x[:, :c["K"]] / (1.0 + torch.exp(-x[:, :c["K"]])) * x[:, c["K"]:]
        q, scale = _mx_quantize(x)
        a = (q.view(x.shape[0], -1, MX) * _mx_scale_values(scale)[..., None]).view(q.shape)
        w = _mx_values(s["w"], s["w_scale"])
    if c["op"] == "gemm":
        y = a @ w.t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(dt)
    if c["op"] == "experts":
        # rows of each expert side by side, the shorter segments padded: one batched fp32 product
        rows = c["T"] * c["topk"]
        off = s["offsets"].long()
        longest = int((off[1:] - off[:-1]).max())
        at = off[:-1, None] + torch.arange(longest, device=DEV)
        real = at < off[1:, None]
        src = at.clamp(max=rows - 1)
        if s["row_token"] is not None:
            src = s["row_token"].long()[src]
        y = torch.bmm(a[src], w.transpose(1, 2).contiguous())
        return y[real].to(dt)
    # every token through every expert that some token chose, weighted by 0 where it did not
    ids, weights = _route_plain(s, c)
    hit = torch.unique(ids)
    hit = hit[hit >= 0]
    share = torch.where(ids[None] == hit[:, None, None], weights, 0.0).sum(2)            # [hit, T]
    x = s["x"].float().t().contiguous().expand(hit.numel(), -1, -1).contiguous()
    up = torch.bmm(_values(c["fmt"], s["w13"][hit], s["w13_scale"][hit]), x)              # [hit, 2I, T]
    gate, up = up[:, :c["I"]], up[:, c["I"]:]
    mid = gate / (1.0 + torch.exp(-gate)) * up * share[:, None]
    y = torch.bmm(_values(c["fmt"], s["w2"][hit], s["w2_scale"][hit]), mid.contiguous()).sum(0).t()
    return (y if s["add"] is None else y + s["add"].float()).to(dt).contiguous()


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_mx(v):
    """The MXFP4 values nearest to v (64 bits, [rows, K]), and their scales."""
    b = v.view(v.shape[0], -1, MX)
    amax = b.abs().amax(2)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 2.0
    scale = torch.where(amax > 0, torch.exp2(e.clamp(min=-127.0)), 2.0 ** -127)
    a = (b / scale[..., None]).abs()
    grid = torch.tensor(E2M1, device=v.device, dtype=torch.float64)
    up = torch.zeros_like(a, dtype=torch.long)
    for k in range(7):                               # a border goes to the value whose code is even
        border = (grid[k] + grid[k + 1]) / 2
        up += (a > border) if k % 2 == 0 else (a >= border)
    return (torch.sign(b) * grid[up] * scale[..., None]).view(v.shape), scale


def _exact_weight(fmt, w, scale):
    """One weight matrix [N, K] in 64 bits."""
    if fmt == "fp8_block":
        N, K = w.shape
        row, col = torch.arange(N, device=w.device) // BLOCK, torch.arange(K, device=w.device) // BLOCK
        return w.double() * scale.double()[row][:, col]
    low, high = (w & 15).long(), ((w >> 4) & 15).long()
    code = torch.stack([low, high], 2).view(w.shape[0], -1)
    K = code.shape[1]
    if fmt == "mxfp4":
        grid = torch.tensor(E2M1, device=w.device, dtype=torch.float64)
        q = torch.where(code >= 8, -1.0, 1.0) * grid[code % 8]
        return q * torch.exp2(scale.double() - 127.0)[:, torch.arange(K, device=w.device) // MX]
    return (code - 16 * (code >= 8)).double() * scale.double().t()[:, torch.arange(K, device=w.device) // BLOCK]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "quant":
        values = torch.empty((c["M"], c["K"]), dtype=torch.float32, device=DEV)     # 3 bits each: exact in fp32
        scales = torch.full((c["M"], 4 * ceil_div(c["K"], BLOCK)), 2.0 ** -127, dtype=torch.float64, device=DEV)
        for r in range(0, c["M"], 512):
            v, sc = _exact_mx(s["x"][r:r + 512].double())
            values[r:r + 512] = v.float()
            scales[r:r + 512, :sc.shape[1]] = sc
        return values, scales
    if c["op"] == "gemm":
        y = _exact_mx(s["x"].double())[0] @ _exact_weight("mxfp4", s["w"], s["w_scale"]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "experts":
        x = s["x"].double()
        if c["gated"]:
            x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
        a = torch.cat([_exact_mx(part)[0] for part in x.split(2048)])
        ends, out = s["offsets"].tolist(), []
        for e in range(c["E"]):
            rows = slice(ends[e], ends[e + 1])
            pick = rows if s["row_token"] is None else s["row_token"][rows].long()
            out.append(a[pick] @ _exact_weight("mxfp4", s["w"][e], s["w_scale"][e]).t())
        return torch.cat(out)
    # routing, token by token
    E, T = c["E"], c["T"]
    x = s["logits"].cpu().double()
    bias = None if s["bias"] is None else s["bias"].cpu().double()
    p = torch.nan_to_num(torch.softmax(x, 1), nan=0.0) if c["score"] == "softmax" else torch.sigmoid(x)
    worth = (p if bias is None else p + bias).masked_fill(x == -math.inf, -math.inf)
    by = x.clone() if bias is None else worth.clone()
    if c["groups"] > 1:
        n = E // c["groups"]
        top = worth.view(T, c["groups"], n).topk(min(c["group_top"], n), dim=2).values
        value = top.nan_to_num(neginf=0.0).sum(2).masked_fill(top[..., 0] == -math.inf, -math.inf)
        place = torch.argsort(torch.argsort(-value, dim=1, stable=True), dim=1)
        by.view(T, c["groups"], n)[place >= c["topk_groups"]] = -math.inf
    ids = torch.argsort(-by, dim=1, stable=True)[:, :c["topk"]]
    w = p.gather(1, ids).masked_fill(by.gather(1, ids) == -math.inf, 0.0)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    w = w * c["scale"]
    y = torch.zeros((T, c["H"]), dtype=torch.float64, device=DEV)
    for e in range(E):
        share = torch.where(ids == e, w, 0.0).sum(1).to(DEV)
        tokens = torch.nonzero(share)[:, 0]
        if not tokens.numel():
            continue
        up = s["x"][tokens].double() @ _exact_weight(c["fmt"], s["w13"][e], s["w13_scale"][e]).t()
        mid = up[:, :c["I"]] * torch.sigmoid(up[:, :c["I"]]) * up[:, c["I"]:]
        y[tokens] += share[tokens, None] * (mid @ _exact_weight(c["fmt"], s["w2"][e], s["w2_scale"][e]).t())
    return y if s["add"] is None else y + s["add"].double()
