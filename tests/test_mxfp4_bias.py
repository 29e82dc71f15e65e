"""The bias of the MXFP4 products lies anywhere that its type allows: a part of a longer vector gives, in every form of the
product, what the same numbers give on their own."""
import ctypes

import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops
from oracle import mxfp4 as O

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def matrix(r, rows, K):
    codes = r.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    scales = np.zeros((rows, O.row_scales(K)), dtype=np.uint8)
    scales[:, :K // 32] = r.integers(120, 128, (rows, K // 32))
    return codes, scales


# rows streamed; tiles of 64 or 128 rows; split tiles; tiles of 256 rows
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(4, 264, 512), (100, 520, 288), (100, 264, 8192), (3590, 3528, 352)])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("offset", [1, 2, 3, 7])
def test_a_part_of_a_longer_vector(M, N, K, dt, offset):
    r = np.random.default_rng([M, N, K])
    (a, sa), (w, sw) = [tuple(torch.from_numpy(t).to(DEV) for t in matrix(r, n, K)) for n in (M, N)]
    # what lies around the part must not be seen
    whole = torch.full((N + 16,), torch.nan, dtype=DT[dt], device=DEV)
    bias = whole[offset:offset + N]
    bias.copy_(torch.from_numpy(r.standard_normal(N) * 8).to(DEV))
    print("bias", M, N, K, dt, offset, flush=True)
    got = ops.w4_mxfp4_gemm(a, sa, w, sw, bias=bias, out_dtype=DT[dt])
    assert torch.equal(got, ops.w4_mxfp4_gemm(a, sa, w, sw, bias=bias.clone(), out_dtype=DT[dt]))
    plain = O.dequantize(a[:3].cpu().numpy(), sa[:3].cpu().numpy()) @ O.dequantize(w.cpu().numpy(), sw.cpu().numpy()).T
    want = plain + bias.double().cpu().numpy()
    size = np.abs(O.dequantize(a[:3].cpu().numpy(), sa[:3].cpu().numpy())) @ np.abs(O.dequantize(w.cpu().numpy(), sw.cpu().numpy())).T
    # one rounding to the output type, and at most one to fp32 for every term and the bias
    tol = np.abs(want) * torch.finfo(DT[dt]).eps / 2 + (K + 2) * 2.0 ** -24 * (size + np.abs(bias.double().cpu().numpy()))
    assert (np.abs(got[:3].double().cpu().numpy() - want) <= tol).all()
    if dt != "f32":
        x = torch.from_numpy(r.standard_normal((M, K))).to(DEV, DT[dt])
        assert torch.equal(ops.w4_mxfp4_linear(x, w, sw, bias=bias), ops.w4_mxfp4_linear(x, w, sw, bias=bias.clone()))


def test_a_bias_between_two_values_is_refused():
    import os
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    L, p = ops.lib(), ctypes.c_void_p
    for dt, at in ((1, 257), (2, 259), (3, 258), (3, 257)):
        assert L.w4_mxfp4_gemm(p(256), p(256), p(256), p(256), p(at), p(256), dt, 4, 256, 256, None, 0, None) == -2
        assert "bias" in L.w4_last_error().decode()
    assert L.w4_mxfp4_linear(p(256), 1, p(256), p(256), p(257), p(256), 4, 256, 256, None, 0, None) == -2
