"""MXFP4 and the layer for a few tokens on the host: what their entry points
refuse (before any launch), workspace sizes, and hand-worked values of the 64-bit
definitions."""
import ctypes

import numpy as np
import pytest

from oracle import mxfp4 as O

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


def test_quantize_refusals(L):
    def q(x=256, dt=1, M=4, K=128, ldx=None, act=0, codes=256, scales=256):
        return L.w4_mxfp4_quantize(p(x), dt, M, K, K if ldx is None else ldx, act, p(codes), p(scales), None)
    assert q(dt=4) == -4 and q(dt=0) == -4
    assert q(M=-1) == -1 and q(K=-32) == -1 and q(act=2) == -1
    assert q(K=48) == -2 and "K=48" in _err(L)
    assert q(ldx=120) == -2 and q(ldx=132) == -2 and q(ldx=248, act=1) == -2
    assert q(dt=3, ldx=130) == -2
    assert q(x=264) == -2 and q(codes=264) == -2 and q(scales=258) == -2
    assert q(x=None) == -1 and q(codes=None) == -1 and q(scales=None) == -1
    assert q(M=1 << 31) == -5 and q(K=1 << 25) == -5 and q(M=1 << 30, K=1 << 20) == -5
    assert q(x=None, M=0) == 0 and q(x=None, K=0) == 0


def test_dequantize_refusals(L):
    def d(codes=256, scales=256, M=4, K=128, out=256, dt=1):
        return L.w4_mxfp4_dequantize(p(codes), p(scales), M, K, p(out), dt, None)
    assert d(dt=5) == -4 and d(M=-1) == -1 and d(K=100) == -2
    assert d(codes=264) == -2 and d(out=264) == -2 and d(scales=257) == -2
    assert d(codes=None) == -1 and d(scales=None) == -1 and d(out=None) == -1
    assert d(M=1 << 31) == -5
    assert d(codes=None, M=0) == 0


def test_gemm_refusals(L):
    def g(a=256, sa=256, w=256, sw=256, out=256, dt=1, M=4, N=256, K=256, ws=None, wsb=0):
        return L.w4_mxfp4_gemm(p(a), p(sa), p(w), p(sw), None, p(out), dt, M, N, K, ws, wsb, None)
    assert g(dt=4) == -4
    assert g(M=-1) == -1 and g(K=0) == -1 and g(N=-8) == -1
    assert g(N=12) == -2 and g(K=40) == -2 and g(K=48) == -2
    assert g(K=(1 << 22) + 32) == -5 and g(M=1 << 31) == -5
    for name in ("a", "w", "out"):
        assert g(**{name: 264}) == -2 and g(**{name: None}) == -1
    for name in ("sa", "sw"):
        assert g(**{name: 258}) == -2 and g(**{name: None}) == -1
    n = ctypes.c_size_t(0)
    assert L.w4_mxfp4_gemm_workspace_bytes(100, 256, 8192, ctypes.byref(n)) == 0 and n.value > 0
    assert g(M=100, K=8192) == -1 and "workspace" in _err(L)
    assert g(M=100, K=8192, ws=p(264), wsb=n.value) == -2
    assert g(a=None, M=0) == 0 and g(a=None, N=0) == 0
    # an output of 2^32 threads or more, whatever the shape's plan
    assert g(M=1 << 30, N=1 << 20) == -5 and g(M=16, N=1 << 29) == -5
    assert L.w4_mxfp4_gemm_workspace_bytes(1, 256, 256, None) == -1


def test_linear_refusals(L):
    def f(x=256, dt=1, w=256, sw=256, out=256, M=4, N=256, K=256, ws=None, wsb=0):
        return L.w4_mxfp4_linear(p(x), dt, p(w), p(sw), None, p(out), M, N, K, ws, wsb, None)
    assert f(dt=3) == -4 and f(K=48) == -2 and f(N=4) == -2 and f(M=-1) == -1
    assert f(x=264) == -2 and f(w=264) == -2 and f(out=264) == -2 and f(sw=258) == -2
    assert f(x=None) == -1 and f(sw=None) == -1
    n = ctypes.c_size_t(9)
    assert L.w4_mxfp4_linear_workspace_bytes(16, 256, 4096, ctypes.byref(n)) == 0 and n.value == 0
    assert L.w4_mxfp4_linear_workspace_bytes(100, 256, 256, ctypes.byref(n)) == 0 and n.value >= 100 * (128 + 8)
    assert f(M=100) == -1 and f(M=100, ws=p(264), wsb=n.value) == -2 and f(M=100, ws=p(256), wsb=n.value - 1) == -1
    assert f(x=None, M=0) == 0


def test_grouped_refusals(L):
    def g(a=256, tok=256, off=256, E=4, w=256, dt=1, T=8, R=64, N=256, K=256, s=256, out=256):
        return L.w4_mxfp4_grouped_gemm(p(a), p(s), p(tok) if tok else None, p(off), E, p(w), p(s), p(out), dt, T, R, N, K, None)
    assert g(dt=3) == -4 and g(K=48) == -2 and g(N=12) == -2 and g(R=-1) == -1
    assert g(E=-1) == -1 and g(E=65536) == -1 and g(T=-1) == -1
    assert g(T=1 << 20, K=4096) == -5 and g(T=0) == -5
    assert g(tok=None) == -1 and "R=64" in _err(L)
    assert g(a=264) == -2 and g(w=264) == -2 and g(out=264) == -2 and g(s=258) == -2
    assert g(off=None) == -1 and g(s=None) == -1
    assert g(R=1 << 30, N=1 << 20, T=1) == -5
    assert g(a=None, R=0) == 0 and g(a=None, E=0) == 0


def test_moe_refusals(L):
    def f(x=256, dt=1, lg=256, ldt=3, ld=None, score=0, G=1, tg=1, gt=1, k=2, fmt=2, w=256, s=256, group=-1, add=None, out=256,
          T=4, E=8, H=256, I=128, ws=256, wsb=1 << 30):
        return L.w4_moe_decode(p(x), dt, p(lg), ldt, E if ld is None else ld, score, None, G, tg, gt, k, 1, 1.0, fmt, p(w), p(s),
                               p(w), p(s), group, p(add) if add else None, p(out), T, E, H, I, p(ws) if ws else None, wsb, None)
    assert f(dt=3) == -4 and f(ldt=4) == -4 and f(fmt=0) == -1 and f(fmt=4) == -1
    assert f(T=-1) == -1 and f(k=9) == -1 and f(E=1032) == -5 and f(E=128, k=65) == -5
    assert f(T=33) == -5 and "T <= 32" in _err(L)
    assert f(H=0) == -1 and f(I=-32) == -1 and f(H=272) == -2 and f(I=48) == -2
    assert f(H=1 << 23) == -5 and f(I=1 << 23) == -5 and f(I=1 << 22, T=32) == -5
    assert f(score=2) == -1 and f(G=3) == -3 and f(G=4, tg=5) == -3 and f(G=4, gt=3) == -5 and f(ld=7) == -2
    assert f(fmt=3, H=160, I=128) == -2 and f(fmt=3, group=64) == -3 and f(fmt=3, group=256) == -3 and f(fmt=3, group=0) == -3
    for name in ("x", "w", "out"):
        assert f(**{name: 264}) == -2 and f(**{name: None}) == -1
    assert f(add=264) == -2 and f(s=260) == -2 and f(s=None) == -1 and f(lg=258) == -2 and f(lg=None) == -1
    assert f(ws=None) == -1 and f(ws=264) == -2 and f(wsb=64) == -1 and "workspace" in _err(L)
    assert f(x=None, T=0) == 0
    n = ctypes.c_size_t(0)
    assert L.w4_moe_decode_workspace_bytes(1, 64, 8, 256, 256, ctypes.byref(n)) == 0 and n.value >= 8 * 256 * 4
    assert L.w4_moe_decode_workspace_bytes(33, 64, 8, 256, 256, ctypes.byref(n)) == -5
    assert L.w4_moe_decode_workspace_bytes(1, 64, 8, 256, 256, None) == -1


def test_python_argument_checks():
    import torch
    from int4_weight_quantized_amd import ops
    u8 = torch.uint8
    c, s = torch.zeros(4, 64, dtype=u8), torch.zeros(4, 4, dtype=u8)
    with pytest.raises(ValueError):
        ops.w4_mxfp4_quantize(torch.zeros(4, 256), act="gelu")
    with pytest.raises(ValueError):
        ops.w4_mxfp4_gemm(c, s, torch.zeros(8, 32, dtype=u8), torch.zeros(8, 4, dtype=u8), out=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="a_scale"):
        ops.w4_mxfp4_gemm(c, s[:, :2], c, s, out=torch.zeros(4, 4))
    with pytest.raises(TypeError):
        ops.w4_mxfp4_gemm(c.int(), s, c, s, out=torch.zeros(4, 4))
    with pytest.raises(ValueError, match="on the GPU"):
        ops.w4_mxfp4_gemm(c, s, c, s, out=torch.zeros(4, 4), workspace=torch.zeros(0, dtype=u8))
    x, lg = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="fmt"):
        ops.w4_moe_decode(x, lg, 2, c, s, c, s, fmt="int8")
    with pytest.raises(ValueError, match="columns"):
        ops.w4_mxfp4_linear(x, torch.zeros(8, 32, dtype=u8), s)


# ------------------------------------------------------------------ hand-worked values

def test_encode_by_hand():
    q = np.array([0.0, 0.25, 0.26, 0.75, 0.76, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 6.0, 99.0, -0.25, -0.3, -5.0, -7.0])
    want = [0, 0, 1, 2, 2, 2, 4, 4, 6, 6, 7, 7, 7, 8, 9, 14, 15]
    assert O.encode(q).tolist() == want
    assert O.decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_quantize_by_hand():
    v = np.zeros((1, 160))
    v[0, 0], v[0, 1] = 7.0, -0.5                           # scale 1: 7 saturates
    v[0, 32] = 2.0 ** -140                                 # below the smallest scale times a step
    v[0, 64], v[0, 65] = 3.0, 1.0                          # scale 1/2: 6 and 2
    v[0, 96] = np.nan
    codes, scales = O.quantize(v)
    assert scales.shape == (1, 8) and scales[0].tolist() == [127, 0, 126, 255, 0, 0, 0, 0]
    assert codes[0, 0] == 7 | 9 << 4 and codes[0, 32] == 7 | 4 << 4 and not codes[0, 48:64].any()
    back = O.dequantize(codes, scales)
    assert back[0, :2].tolist() == [6.0, -0.5] and back[0, 64:66].tolist() == [3.0, 1.0] and np.isnan(back[0, 96:128]).all()


def test_moe_by_hand():
    """One token, two experts of equal score: half of each expert's result."""
    x = np.array([[1.0, 2.0]])
    w13 = np.zeros((2, 2, 2))
    w13[0] = [[1.0, 0.0], [0.0, 1.0]]                      # gate 1, up 2
    w13[1] = [[0.0, 1.0], [1.0, 0.0]]                      # gate 2, up 1
    w2 = np.array([[[1.0], [0.0]], [[0.0], [1.0]]])
    y, _, _ = O.moe(x, np.array([[0.0, 0.0]]), 2, w13, w2, add=np.array([[10.0, 20.0]]))
    silu = lambda z: z / (1 + np.exp(-z))  # noqa: E731
    assert np.allclose(y, [[10 + 0.5 * silu(1.0) * 2.0, 20 + 0.5 * silu(2.0) * 1.0]])
