"""CPU-only: the work memory of the 8-bit linear layer's gradients is what the
header says."""
import ctypes as C

import pytest

import extreme_label_sparse_gb300 as sgpkg

P, OFF2 = C.c_void_p(256), C.c_void_p(258)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    sgpkg.build()
    return sgpkg.load()


@pytest.mark.parametrize("T,H,N", [(1, 64, 1 << 24), (3, 1 << 20, 300), (128, 4096, 131072), (512, 4096, 4096),
                                   (8192, 4096, 4096), (65536, 1001, 16001), (1 << 24, 64, 70)])
def test_backward_work_memory_is_bounded(lib, T, H, N):
    n = C.c_int64(-1)
    ldh, ldn = -(-H // 16) * 16, -(-N // 8) * 8
    for dout, copy in ((P, 0), (OFF2, 2 * T * ldn)):
        assert lib.sg_linear8_work(P, ldh, T, H, P, ldh, N, dout, ldn, 1, C.byref(n)) == 0
        # parts: 4 x 152 tiles of 128 x 256 fp32 for each product
        assert 2 * ldh * max(T, N) <= n.value <= 2 * ldh * (T + N) + copy + 2 * 4 * 152 * 131072 + 4096
