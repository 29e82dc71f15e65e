"""A routed-expert layer on the FP8 expert path: router logits and hidden rows in, the experts' weighted sum out.

    route -> quantize rows -> gate/up product over the experts -> SwiGLU + quantize -> down product -> combine

Weights are E4M3 with one fp32 scale per 128 x 128 block (the weight_block_size [128, 128] of W4AFP8Config.from_config).
Every buffer is allocated once for `max_tokens`, so a call allocates nothing and can be captured into a graph.

    python -m int4_weight_quantized_amd.fp8_experts        # times the layer at a few token counts
"""
from __future__ import annotations

import torch

from . import ops


class Fp8Experts:
    """w13 [E, 2 I, H] (gate rows, then up rows) and w2 [E, H, I] E4M3 codes, w13_scale [E, ceil(2I/128), ceil(H/128)] and
    w2_scale [E, ceil(H/128), ceil(I/128)] fp32. `routing` goes to ops.w4_route (score, bias, n_groups, ...). Up to
    `decode_tokens` tokens (at most W4_MOE_DECODE_MAX_TOKENS) run as one call, ops.w4_moe_decode, which does not quantize
    the activations: none unless asked for."""

    def __init__(self, w13, w13_scale, w2, w2_scale, topk: int, max_tokens: int, dtype=torch.bfloat16,
                 decode_tokens: int = 0, **routing):
        E, H, I = w2.shape
        if tuple(w13.shape) != (E, 2 * I, H):
            raise ValueError(f"w13 must be [{E}, {2 * I}, {H}] for w2 {tuple(w2.shape)}, got {tuple(w13.shape)}")
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
        self._ids, self._weights = buf(max_tokens, topk, dt=i32), buf(max_tokens, topk, dt=f32)
        self._row_token, self._offsets, self._row_of = buf(rows, dt=i32), buf(E + 1, dt=i32), buf(max_tokens, topk, dt=i32)
        self._x, self._xs = buf(max_tokens, H, dt=u8), buf(max_tokens, -(-H // 128), dt=f32)
        self._h = buf(rows, 2 * I, dt=dtype)
        self._a, self._as = buf(rows, I, dt=u8), buf(rows, -(-I // 128), dt=f32)
        self._y = buf(rows, H, dt=dtype)
        self._ws = ops.w4_route_workspace(max_tokens, E, topk, device=dev)
        if self.decode_tokens:
            self._decode_ws = ops.w4_moe_decode_workspace(self.decode_tokens, E, topk, H, I, device=dev)

    def __call__(self, x, logits, add=None, out=None, stream=None):
        """x [T, H] in the layer's type, logits [T, E] -> [T, H] (+ add [T, H]). The layer's buffers are reused by the
        next call: calls on different streams must not overlap."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens exceed max_tokens={self.max_tokens}")
        if self.decode_tokens and x.dtype != self.dtype:     # the same types on both sides of decode_tokens
            raise TypeError(f"x must be {self.dtype}, the layer's type, got {x.dtype}")
        if T and T <= self.decode_tokens:
            return ops.w4_moe_decode(x, logits, self.topk, self.w13, self.w13_scale, self.w2, self.w2_scale, add=add, out=out,
                                     workspace=self._decode_ws, stream=stream, **self.routing)
        R = T * self.topk
        plan = (self._ids[:T], self._weights[:T], self._row_token[:R], self._offsets, self._row_of[:T])
        _, weights, row_token, offsets, row_of = ops.w4_route(
            logits, self.topk, out=plan, workspace=self._ws, stream=stream, **self.routing)
        xq, xs = ops.w4_fp8_block_quantize(x, out=(self._x[:T], self._xs[:T]), stream=stream)
        h = ops.w4_fp8_block_grouped_gemm(xq, xs, row_token, offsets, self.w13, self.w13_scale, out=self._h[:R],
                                          stream=stream)
        # rows past the last planned one (tokens without an expert) hold leftovers, which no token reads
        aq, asc = ops.w4_fp8_block_quantize(h, act="swiglu", out=(self._a[:R], self._as[:R]), stream=stream)
        y = ops.w4_fp8_block_grouped_gemm(aq, asc, None, offsets, self.w2, self.w2_scale, out=self._y[:R],
                                          stream=stream)
        return ops.w4_combine(y, row_of, weights, add=add, out=out, stream=stream)


def random_experts(E: int, H: int, I: int, topk: int, max_tokens: int, seed: int = 0, **kw) -> Fp8Experts:
    """A layer with random weights of the usual spread."""
    g = torch.Generator("cuda").manual_seed(seed)

    def weights(n, k):
        w = (torch.randn((E, n, k), device="cuda", generator=g) * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s = torch.rand((E, -(-n // 128), -(-k // 128)), device="cuda", generator=g) * 2e-4 + 1e-4
        return w, s
    return Fp8Experts(*weights(2 * I, H), *weights(H, I), topk, max_tokens, **kw)


def main():
    E, H, I, topk = 64, 7168, 2048, 8
    layer = random_experts(E, H, I, topk, 8192)
    decode = Fp8Experts(layer.w13, layer.w13_scale, layer.w2, layer.w2_scale, topk, 32, decode_tokens=32)
    for layer, T in [(layer, T) for T in (1, 8, 64, 512, 8192)] + [(decode, T) for T in (1, 8, 32)]:
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
        print(f"{T} tokens{', activations not quantized' if layer is decode else ''}: {start.elapsed_time(end) * 100:.0f} us  "
              f"({E} experts, hidden {H}, intermediate {I}, top {topk})", flush=True)


if __name__ == "__main__":
    main()
