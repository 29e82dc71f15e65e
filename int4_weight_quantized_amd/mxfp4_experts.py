"""A routed-expert layer on MXFP4 weights: router logits and hidden rows in, the experts' weighted sum out.

Few tokens (a decode step) run as one call, weight-only (ops.w4_moe_decode); more run in stages, activations in MXFP4 too:

    route -> quantize rows -> gate/up product over the experts -> SwiGLU + quantize -> down product -> combine

Every buffer is allocated once for `max_tokens`, so a call allocates nothing and can be captured into a graph.

    python -m int4_weight_quantized_amd.mxfp4_experts        # times the layer at a few token counts
"""
from __future__ import annotations

import torch

from . import ops


class Mxfp4Experts:
    """w13 uint8 [E, 2 I, H / 2] (gate rows, then up rows) and w2 [E, H, I / 2] codes, w13_scale uint8
    [E, 2 I, 4 ceil(H / 128)] and w2_scale [E, H, 4 ceil(I / 128)], as ops.w4_mxfp4_quantize lays them out. `routing` goes
    to ops.w4_route (score, bias, n_groups, ...). Up to `decode_tokens` tokens (at most W4_MOE_DECODE_MAX_TOKENS) take the
    one call; its activations are not quantized, so the two paths differ by the quantization. The default prefers
    that to time: the one call is the faster up to about 12 tokens. (64 experts, 8 chosen, of 7168 x 2048: 1 token 44 us in
    one call and 56 in stages, 8 tokens 187 and 194, 12 tokens 225 and 233, 16 tokens 258 and 253, 32 tokens 324 and 281;
    of 2048 x 1024: 17 and 29, 46 and 49, 54 and 54, 62 and 55, 80 and 58.)"""

    def __init__(self, w13, w13_scale, w2, w2_scale, topk: int, max_tokens: int, dtype=torch.bfloat16,
                 decode_tokens: int = ops.W4_MOE_DECODE_MAX_TOKENS, **routing):
        E, H, I = w2.shape[0], w2.shape[1], 2 * w2.shape[2]
        if tuple(w13.shape) != (E, 2 * I, H // 2):
            raise ValueError(f"w13 must be [{E}, {2 * I}, {H // 2}] for w2 {tuple(w2.shape)}, got {tuple(w13.shape)}")
        if not 0 <= decode_tokens <= ops.W4_MOE_DECODE_MAX_TOKENS:
            raise ValueError(f"decode_tokens={decode_tokens} outside 0..{ops.W4_MOE_DECODE_MAX_TOKENS}")
        dev = w13.device
        self.w13, self.w13_scale, self.w2, self.w2_scale = w13, w13_scale, w2, w2_scale
        self.topk, self.max_tokens, self.dtype, self.routing = topk, max_tokens, dtype, routing
        self.E, self.H, self.I, self.decode_tokens = E, H, I, min(decode_tokens, max_tokens)
        rows = max_tokens * topk

        def buf(*shape, dt):
            return torch.empty(shape, dtype=dt, device=dev)
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        if self.decode_tokens:
            self._decode_ws = ops.w4_moe_decode_workspace(self.decode_tokens, E, topk, H, I, device=dev)
        if max_tokens > self.decode_tokens:
            self._ids, self._weights = buf(max_tokens, topk, dt=i32), buf(max_tokens, topk, dt=f32)
            self._row_token, self._offsets = buf(rows, dt=i32), buf(E + 1, dt=i32)
            self._row_of = buf(max_tokens, topk, dt=i32)
            self._x, self._xs = buf(max_tokens, H // 2, dt=u8), buf(max_tokens, w13_scale.shape[2], dt=u8)
            self._h = buf(rows, 2 * I, dt=dtype)
            self._a, self._as = buf(rows, I // 2, dt=u8), buf(rows, w2_scale.shape[2], dt=u8)
            self._y = buf(rows, H, dt=dtype)
            self._ws = ops.w4_route_workspace(max_tokens, E, topk, device=dev)

    def __call__(self, x, logits, add=None, out=None, stream=None):
        """x [T, H] in the layer's type, logits [T, E] -> [T, H] (+ add [T, H]). The layer's buffers are reused by the
        next call: calls on different streams must not overlap."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens exceed max_tokens={self.max_tokens}")
        if x.dtype != self.dtype:                            # the same types on both sides of decode_tokens
            raise TypeError(f"x must be {self.dtype}, the layer's type, got {x.dtype}")
        if T <= self.decode_tokens:
            return ops.w4_moe_decode(x, logits, self.topk, self.w13, self.w13_scale, self.w2, self.w2_scale, fmt="mxfp4",
                                     add=add, out=out, workspace=self._decode_ws if T else None, stream=stream,
                                     **self.routing)
        R = T * self.topk
        plan = (self._ids[:T], self._weights[:T], self._row_token[:R], self._offsets, self._row_of[:T])
        _, weights, row_token, offsets, row_of = ops.w4_route(
            logits, self.topk, out=plan, workspace=self._ws, stream=stream, **self.routing)
        xq, xs = ops.w4_mxfp4_quantize(x, out=(self._x[:T], self._xs[:T]), stream=stream)
        h = ops.w4_mxfp4_grouped_gemm(xq, xs, row_token, offsets, self.w13, self.w13_scale, out=self._h[:R], stream=stream)
        # rows past the last planned one (tokens without an expert) hold leftovers, which no token reads
        aq, asc = ops.w4_mxfp4_quantize(h, act="swiglu", out=(self._a[:R], self._as[:R]), stream=stream)
        y = ops.w4_mxfp4_grouped_gemm(aq, asc, None, offsets, self.w2, self.w2_scale, out=self._y[:R], stream=stream)
        return ops.w4_combine(y, row_of, weights, add=add, out=out, stream=stream)

    @classmethod
    def from_weights(cls, w13, w2, topk: int, max_tokens: int, **kw) -> "Mxfp4Experts":
        """A layer from w13 [E, 2 I, H] and w2 [E, H, I] in bf16, fp16 or fp32, quantized here."""
        def pack(w):
            E, N, K = w.shape
            codes, scales = ops.w4_mxfp4_quantize(w.reshape(E * N, K))
            return codes.view(E, N, -1), scales.view(E, N, -1)
        return cls(*pack(w13), *pack(w2), topk, max_tokens, **kw)


def random_experts(E: int, H: int, I: int, topk: int, max_tokens: int, seed: int = 0, **kw) -> Mxfp4Experts:
    """A layer with random weights of the usual spread."""
    g = torch.Generator("cuda").manual_seed(seed)

    def weights(n, k):
        codes, scales = [], []
        for _ in range(E):
            c, s = ops.w4_mxfp4_quantize(torch.randn((n, k), device="cuda", generator=g) * 0.02)
            codes.append(c)
            scales.append(s)
        return torch.stack(codes), torch.stack(scales)
    return Mxfp4Experts(*weights(2 * I, H), *weights(H, I), topk, max_tokens, **kw)


def main():
    E, H, I, topk = 64, 7168, 2048, 8
    layer = random_experts(E, H, I, topk, 8192)
    for T in (1, 8, 32, 64, 512, 8192):
        x = torch.randn((T, H), device="cuda").bfloat16()
        logits = torch.randn((T, E), device="cuda")
        out = torch.empty_like(x)
        for _ in range(3):
            layer(x, logits, out=out)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(10):
            layer(x, logits, out=out)
        end.record()
        torch.cuda.synchronize()
        print(f"{T} tokens: {start.elapsed_time(end) * 100:.0f} us  ({E} experts, hidden {H}, intermediate {I}, "
              f"top {topk})", flush=True)


if __name__ == "__main__":
    main()
