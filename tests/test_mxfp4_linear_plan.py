"""Where w4_mxfp4_linear quantizes its rows within the product, and that it makes no difference to the results."""
import ctypes
import os

import numpy as np
import pytest
import torch

from int4_weight_quantized_amd import ops

# as measured: (rows, columns, K, whether one launch is the faster)
PLANS = [(16, 256, 4096, True), (12, 4096, 4096, True), (14, 4096, 4096, True), (16, 4096, 4096, False), (8, 4096, 7168, True),
         (4, 4096, 14336, True), (8, 8192, 4096, True), (12, 8192, 4096, False), (8, 14336, 4096, True), (4, 28672, 4096, True),
         (8, 28672, 4096, False), (17, 256, 32, False)]


@pytest.mark.parametrize("M,N,K,one", PLANS)
def test_one_launch_where_it_is_the_faster(M, N, K, one):
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    n = ctypes.c_size_t(0)
    assert ops.lib().w4_mxfp4_linear_workspace_bytes(M, N, K, ctypes.byref(n)) == 0
    assert (n.value == 0) == one


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,one", PLANS)
def test_both_give_the_same(M, N, K, one):
    r = np.random.default_rng([M, N, K])
    x = torch.from_numpy(r.standard_normal((M, K))).to("cuda", torch.bfloat16)
    w = torch.from_numpy(r.integers(0, 256, (N, K // 2)).astype(np.uint8)).to("cuda")
    s = torch.from_numpy(r.integers(120, 128, (N, 4 * -(-K // 128))).astype(np.uint8)).to("cuda")
    print("plan", M, N, K, flush=True)
    assert torch.equal(ops.w4_mxfp4_linear(x, w, s), ops.w4_mxfp4_gemm(*ops.w4_mxfp4_quantize(x), w, s))
