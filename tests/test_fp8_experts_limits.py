"""The FP8 expert path's size limits on the host: sizes whose launch would need
2^32 threads or more are refused before any launch, the largest below them are
not."""
import ctypes

import pytest

p = ctypes.c_void_p
UNSUPPORTED = -5


@pytest.fixture(scope="module")
def L():
    import os
    from int4_weight_quantized_amd import ops
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return ops.lib()


def test_route_tokens(L):
    n = ctypes.c_size_t()
    last = (1 << 28) - 64                                       # 2^22 - 1 blocks of 1024 threads
    assert L.w4_route_workspace_bytes(last, 8, 2, ctypes.byref(n)) == 0 and n.value > 0
    assert L.w4_route_workspace_bytes(last + 1, 8, 2, ctypes.byref(n)) == UNSUPPORTED
    assert b"2^28 - 64" in L.w4_last_error()
    rc = L.w4_route(p(256), 1, last + 1, 8, 8, 0, None, 1, 1, 1, 1, 1, 1.0, p(256), p(256), p(256), p(256), p(256), p(256),
                    1 << 40, None)
    assert rc == UNSUPPORTED


def test_dense_product_tiles(L):
    """256 threads a tile: 2^24 tiles are refused, by the product and by its workspace size."""
    n = ctypes.c_size_t()

    def both(M, N, K=16):
        """Codes of the workspace size and of the product (null operands: refused later, as invalid)."""
        return (L.w4_fp8_block_gemm_workspace_bytes(M, N, K, ctypes.byref(n)),
                L.w4_fp8_block_gemm(None, None, None, None, None, None, 1, M, N, K, None, 0, None))
    for M, N in ((1, (1 << 29) - 32), (16, (1 << 29) - 32), (64, 1 << 30), (128, 1 << 30), (1 << 30, 128)):
        assert both(M, N) == (0, -1), (M, N)
    for M, N in ((1, 1 << 29), (16, 1 << 29), (256, 1 << 30), (1 << 30, 256), (1 << 27, 2048)):
        assert both(M, N) == (UNSUPPORTED, UNSUPPORTED), (M, N)
    assert both(1 << 30, 256)[1] == UNSUPPORTED and b"threads" in L.w4_last_error()


def test_grouped_product_tiles(L):
    def g(E, R, N, K=16):
        return L.w4_fp8_block_grouped_gemm(p(256), p(256), p(256), p(256), E, p(256), p(256), None, 1, 8, R, N, K, None)
    # streamed, 16 x 32: (65535 / 16 + 65535) * N / 32 blocks of 256 threads
    assert g(65535, 65535, 7680) == -1
    assert g(65535, 65535, 7688) == UNSUPPORTED and b"threads" in L.w4_last_error()
    # 128 x 128: (2^30 / 128 + 1) blocks of 256; 256 x 256: (2^30 / 256 + 1) * N / 256 of 512
    assert g(1, 1 << 30, 128) == -1 and g(1, 1 << 30, 256) == -1
    assert g(1, 1 << 30, 512) == UNSUPPORTED
