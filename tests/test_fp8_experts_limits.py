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
