"""The expert layers as a user runs them: Mxfp4Experts' two paths (one call for few tokens, stages for many) against the
operators called one by one, and Fp8Experts with and without the one call."""
import pytest
import torch

from int4_weight_quantized_amd import ops
from int4_weight_quantized_amd.fp8_experts import Fp8Experts, random_experts as fp8_layer
from int4_weight_quantized_amd.mxfp4_experts import Mxfp4Experts, random_experts

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(T, H, E, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return (torch.randn((T, H), device=DEV, generator=g).bfloat16(), torch.randn((T, E), device=DEV, generator=g))


@pytest.mark.parametrize("T", [0, 1, 8, 9, 70])
def test_mxfp4_layer_is_its_operators(T):
    E, H, I, topk = 8, 416, 160, 3
    routing = dict(score="sigmoid", scale=1.5)
    layer = random_experts(E, H, I, topk, 80, decode_tokens=8, **routing)
    x, logits = inputs(T, H, E, T)
    got = layer(x, logits, add=x)
    if T <= 8:
        want = ops.w4_moe_decode(x, logits, topk, layer.w13, layer.w13_scale, layer.w2, layer.w2_scale, fmt="mxfp4", add=x,
                                 **routing)
    else:
        ids, weights, row_token, offsets, row_of = ops.w4_route(logits, topk, **routing)
        h = ops.w4_mxfp4_grouped_gemm(*ops.w4_mxfp4_quantize(x), row_token, offsets, layer.w13, layer.w13_scale)
        y = ops.w4_mxfp4_grouped_gemm(*ops.w4_mxfp4_quantize(h, act="swiglu"), None, offsets, layer.w2, layer.w2_scale)
        want = ops.w4_combine(y, row_of, weights, add=x)
    assert torch.equal(got, want)


def test_from_weights():
    g = torch.Generator(DEV).manual_seed(1)
    w13, w2 = (torch.randn(s, device=DEV, generator=g) * 0.05 for s in ((4, 128, 96), (4, 96, 64)))
    layer = Mxfp4Experts.from_weights(w13.bfloat16(), w2.bfloat16(), 2, 8)
    for e in range(4):
        codes, scales = ops.w4_mxfp4_quantize(w13[e].bfloat16())
        assert torch.equal(layer.w13[e], codes) and torch.equal(layer.w13_scale[e], scales)
    x, logits = inputs(3, 96, 4, 2)
    assert layer(x, logits).isfinite().all()


def test_fp8_layer_with_the_one_call():
    E, H, I, topk = 8, 256, 128, 2
    layer = fp8_layer(E, H, I, topk, 64)
    w = (layer.w13, layer.w13_scale, layer.w2, layer.w2_scale)
    few = Fp8Experts(*w, topk, 64, decode_tokens=4)
    for T in (0, 4, 5):
        x, logits = inputs(T, H, E, T)
        want = ops.w4_moe_decode(x, logits, topk, *w) if 0 < T <= 4 else layer(x, logits)
        assert torch.equal(few(x, logits), want)


def test_layers_refuse():
    layer = random_experts(4, 64, 32, 2, 8)
    x, logits = inputs(9, 64, 4, 0)
    with pytest.raises(ValueError, match="max_tokens"):
        layer(x, logits)
    w = (layer.w13, layer.w13_scale, layer.w2, layer.w2_scale)
    with pytest.raises(ValueError, match="decode_tokens"):
        Mxfp4Experts(*w, 2, 64, decode_tokens=33)
    with pytest.raises(ValueError, match="w13"):
        Mxfp4Experts(w[0][:, :32], *w[1:], 2, 64)


@pytest.mark.parametrize("T", [2, 40])
def test_mxfp4_layer_captured(T):
    E, H, I, topk = 8, 256, 128, 2
    layer = random_experts(E, H, I, topk, 64)
    x, logits = inputs(T, H, E, 1)
    out = torch.empty_like(x)
    layer(x, logits, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out=out)
    other = random_experts(E, H, I, topk, 64)
    for k in range(4):
        nx, nl = inputs(T, H, E, 10 + k)
        x.copy_(nx)
        logits.copy_(nl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other(x, logits)), k
