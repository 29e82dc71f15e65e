"""The FP8 expert path on the host: what its entry points refuse (before any
launch), and hand-worked values of the 64-bit definitions."""
import ctypes

import numpy as np
import pytest

from oracle import fp8_experts as O
from oracle.w4_oracle import e4m3_decode

p = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    import os
    from int4_weight_quantized_amd import ops
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return ops.lib()


def _err(L):
    return L.w4_last_error().decode()


def _route(L, x=256, dt=3, T=4, E=8, ld=None, score=0, bias=None, G=1, tg=1, gt=1, k=2, ptr=256, ws=None, wsb=0):
    return L.w4_route(p(x), dt, T, E, E if ld is None else ld, score, bias, G, tg, gt, k, 1, 1.0, p(ptr), p(ptr), p(ptr),
                      p(ptr), p(ptr), ws, wsb, None)


def test_route_refusals(L):
    assert _route(L, dt=4) == -4
    assert _route(L, T=-1) == -1 and _route(L, E=0) == -1 and _route(L, k=0) == -1
    assert _route(L, k=9) == -1 and "topk=9 exceeds E=8" in _err(L)
    assert _route(L, E=1032) == -5 and _route(L, E=128, k=65) == -5
    assert _route(L, T=1 << 30, k=2) == -5                     # T * topk reaches 2^31
    assert _route(L, score=2) == -1
    assert _route(L, G=3) == -3 and _route(L, G=0) == -3 and _route(L, E=130, G=65) == -3
    assert _route(L, G=4, tg=5) == -3 and _route(L, G=4, tg=0) == -3
    assert _route(L, G=4, gt=3) == -5
    assert _route(L, ld=7) == -2
    assert _route(L, x=None) == -1 and _route(L, ptr=None) == -1
    assert _route(L, x=258) == -2                              # fp32 logits on a 2-byte boundary
    rc = _route(L, T=65, ws=None)
    assert rc == -1 and "workspace" in _err(L)
    assert _route(L, T=65, ws=p(264), wsb=1 << 20) == -2


def test_route_workspace_sizes(L):
    n = ctypes.c_size_t(7)
    assert L.w4_route_workspace_bytes(1, 64, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert L.w4_route_workspace_bytes(1 << 20, 256, 8, ctypes.byref(n)) == 0 and n.value > 0
    assert L.w4_route_workspace_bytes(4, 8, 9, ctypes.byref(n)) == -1
    assert L.w4_route_workspace_bytes(4, 8, 2, None) == -1


def test_block_quantize_refusals(L):
    q = L.w4_fp8_block_quantize
    assert q(p(256), 3, 4, 128, 128, 0, p(256), p(256), None) == -4           # fp32 activations
    assert q(p(256), 1, -1, 128, 128, 0, p(256), p(256), None) == -1
    assert q(p(256), 1, 4, 12, 16, 0, p(256), p(256), None) == -2             # K % 8
    assert q(p(256), 1, 4, 128, 120, 0, p(256), p(256), None) == -2           # ldx < K
    assert q(p(256), 1, 4, 128, 248, 1, p(256), p(256), None) == -2           # ldx < 2K with the gate
    assert q(p(256), 1, 4, 128, 132, 0, p(256), p(256), None) == -2           # ldx % 8
    assert q(p(256), 1, 4, 128, 128, 2, p(256), p(256), None) == -1           # activation
    assert q(p(264), 1, 4, 128, 128, 0, p(256), p(256), None) == -2
    assert q(p(256), 1, 4, 128, 128, 0, p(260), p(256), None) == -2
    assert q(None, 1, 4, 128, 128, 0, p(256), p(256), None) == -1
    assert q(p(256), 1, 4, 1 << 25, 1 << 25, 0, p(256), p(256), None) == -5
    assert q(None, 1, 0, 128, 128, 0, None, None, None) == 0 and q(None, 1, 4, 0, 0, 0, None, None, None) == 0


def test_block_gemm_refusals(L):
    def g(M=4, N=128, K=256, dt=1, a=256, asc=256, w=256, wsc=256, out=256, ws=1 << 20, wsb=1 << 40):
        return L.w4_fp8_block_gemm(p(a), p(asc), p(w), p(wsc), None, p(out), dt, M, N, K, p(ws), wsb, None)
    assert g(dt=4) == -4
    assert g(M=-1) == -1 and g(K=0) == -1
    assert g(N=12) == -2 and "output N=12" in _err(L)
    assert g(K=24) == -2 and "multiple of 16" in _err(L)
    assert g(M=1 << 31) == -5
    for name in ("a", "asc", "w", "wsc", "out"):
        assert g(**{name: None}) == -1, name
    for name in ("a", "w", "out"):
        assert g(**{name: 264}) == -2, name
    assert L.w4_fp8_block_gemm(None, None, None, None, None, None, 1, 0, 128, 256, None, 0, None) == 0
    assert L.w4_fp8_block_gemm(None, None, None, None, None, None, 1, 4, 0, 256, None, 0, None) == 0
    n = ctypes.c_size_t()
    assert L.w4_fp8_block_gemm_workspace_bytes(4, 128, 24, ctypes.byref(n)) == -2
    assert L.w4_fp8_block_gemm_workspace_bytes(4, 128, 256, None) == -1
    # a workspace one byte short is refused wherever one is needed
    for M, N, K in ((1, 4096, 16384), (64, 2048, 16384), (200, 4096, 14336)):
        assert L.w4_fp8_block_gemm_workspace_bytes(M, N, K, ctypes.byref(n)) == 0
        if n.value:
            assert g(M=M, N=N, K=K, wsb=n.value - 1) == -1 and "workspace" in _err(L)
            assert g(M=M, N=N, K=K, ws=264) == -2


def test_grouped_gemm_refusals(L):
    def g(T=8, R=16, N=128, K=256, E=4, dt=1, a=256, asc=256, rt=256, off=256, w=256, wsc=256, out=256):
        return L.w4_fp8_block_grouped_gemm(p(a), p(asc), p(rt), p(off), E, p(w), p(wsc), p(out), dt, T, R, N, K, None)
    assert g(dt=3) == -4 and g(dt=4) == -4
    assert g(E=-1) == -1 and g(E=65536) == -1 and g(T=-1) == -1 and g(R=-1) == -1
    assert g(N=12) == -2 and g(K=24) == -2
    assert g(T=1 << 23, K=256) == -5                            # T * K reaches 2^31
    assert g(rt=None, T=8, R=16) == -1 and "R=16" in _err(L)
    for name in ("a", "asc", "off", "w", "wsc", "out"):
        assert g(**{name: None}) == -1, name
    for name in ("a", "w", "out"):
        assert g(**{name: 264}) == -2, name
    assert g(R=0) == 0 and g(N=0) == 0 and g(E=0) == 0


def test_combine_refusals(L):
    def c(T=4, R=8, k=2, N=64, dt=1, y=256, ro=256, wt=256, add=None, out=256):
        return L.w4_combine(p(y), dt, p(ro), p(wt), p(add), p(out), T, R, k, N, None)
    assert c(dt=5) == -4
    assert c(T=-1) == -1 and c(R=-1) == -1 and c(k=0) == -1 and c(N=-8) == -1
    assert c(N=12) == -2
    assert c(k=1025) == -5
    for name in ("y", "ro", "wt", "out"):
        assert c(**{name: None}) == -1, name
    for name in ("y", "add", "out"):
        assert c(**{name: 264}) == -2, name
    assert c(T=0) == 0 and c(N=0) == 0


def test_python_argument_checks():
    import torch
    from int4_weight_quantized_amd import ops
    x = torch.zeros((4, 256), dtype=torch.uint8)
    s = torch.zeros((4, 2))
    w = torch.zeros((128, 256), dtype=torch.uint8)
    ws = torch.zeros((1, 2))
    with pytest.raises(TypeError, match="E4M3"):
        ops.w4_fp8_block_gemm(x.float(), s, w, ws)
    with pytest.raises(ValueError, match="columns"):
        ops.w4_fp8_block_gemm(x[:, :128], s, w, ws)
    with pytest.raises(ValueError, match="a_scale"):
        ops.w4_fp8_block_gemm(x, s[:, :1], w, ws)
    with pytest.raises(TypeError, match="w_scale"):
        ops.w4_fp8_block_gemm(x, s, w, ws.double())
    with pytest.raises(ValueError, match="GPU"):
        ops.w4_route(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError, match="act"):
        ops.w4_fp8_block_quantize(torch.zeros((4, 8), dtype=torch.bfloat16), act="gelu")


# ---- the definitions, on values worked out by hand

def test_route_by_hand():
    x = np.array([[0.0, 2.0, 2.0, -np.inf], [np.nan, -np.inf, np.nan, -np.inf], [1.0, 1.0, 1.0, 1.0]])
    ids, w = O.route(x, 2)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 1]] and np.allclose(w, [[0.5, 0.5], [0, 0], [0.5, 0.5]])
    # the bias moves the choice and not the weight: sigmoid(0) = 1/2
    ids, w = O.route([[0.0, 0.0, 0.0, 0.0]], 2, score="sigmoid", bias=[0, .1, .3, .2], renorm=False, scale=2.5)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[1.25, 1.25]])
    # groups {0,1}, {2,3}: by the best one group 1 wins, by the best two group 0
    x = [[1.0, 0.9, 1.2, -9.0]]
    assert O.route(x, 1, score="sigmoid", n_groups=2, group_top=1)[0].tolist() == [[2]]
    assert O.route(x, 1, score="sigmoid", n_groups=2, group_top=2)[0].tolist() == [[0]]
    row_token, off, row_of = O.plan(np.array([[2, 0], [0, -1], [2, 1]], dtype=np.int32), 4)
    assert off.tolist() == [0, 2, 3, 5, 5] and row_token.tolist() == [0, 1, 2, 0, 2, -1]
    assert row_of.tolist() == [[3, 0], [1, -1], [4, 2]]


def test_quantize_and_products_by_hand():
    v = np.zeros((1, 130), dtype=np.float32)
    v[0, 0], v[0, 1], v[0, 129] = 448.0, -3.3, 7.0
    codes, s = O.block_quantize(v)
    assert s.tolist() == [[1.0, np.float32(7.0) / np.float32(448.0)]]
    assert e4m3_decode(codes)[0, [0, 1, 129]].tolist() == [448.0, -3.25, 448.0]
    a = np.zeros((1, 144), dtype=np.uint8)
    w = np.zeros((8, 144), dtype=np.uint8)
    a[0, 0] = a[0, 140] = 0x38                                  # 1.0
    w[3, 0], w[3, 140] = 0x40, 0x44                             # 2.0, 3.0
    y, mag = O.block_gemm(a, np.array([[2.0, 10.0]]), w, np.array([[0.5, 0.25]]), bias=np.ones(8))
    assert y[0, 3] == 2 * 0.5 * 2 + 10 * 0.25 * 3 + 1 and y[0, 2] == 1 and mag[0, 3] == y[0, 3]
    out, _ = O.combine(np.array([[1.0], [10.0]]), np.array([[1, -1], [0, 1]]), np.array([[.5, 9.], [2., .25]]))
    assert out.tolist() == [[5.0], [4.5]]
    assert np.allclose(O.silu_gate([[0.0, 2.0, 5.0, -1.0]]), [[0.0, -2.0 / (1 + np.exp(-2.0))]])
