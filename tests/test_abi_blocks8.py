"""CPU-only checks of the calls for blocks on 8-bit integers: bad arguments are
refused before anything is launched, and work sizes need no GPU."""
import ctypes as C

import pytest

import extreme_label_sparse_gb300 as sgpkg

P = C.c_void_p(256)  # never dereferenced: validation fails first
OFF1, OFF2 = C.c_void_p(257), C.c_void_p(258)
INVALID, UNSUPPORTED = sgpkg.SG_ERR_INVALID, sgpkg.SG_ERR_UNSUPPORTED
BF, F16, F32, E4M3 = sgpkg.SG_BF16, sgpkg.SG_F16, sgpkg.SG_F32, sgpkg.SG_E4M3


@pytest.fixture(scope="module")
def lib():
    sgpkg.build()
    return sgpkg.load()


def refused(call, ok, cases):
    for at, bad, want in cases:
        args = list(ok)
        args[at] = bad
        assert call(*args) == want, (call.__name__, at, bad, sgpkg.last_error())
        assert call.__name__ in sgpkg.last_error()


def test_pack_refusals(lib):
    refused(lib.sg_pack8, [P, 8, 4, 8, BF, 128, P, 8, P, None],
            ((0, None, INVALID), (6, None, INVALID), (8, None, INVALID), (1, 7, INVALID), (7, 7, INVALID),
             (2, -1, INVALID), (3, 0, INVALID), (4, E4M3, INVALID), (4, 9, INVALID), (5, 64, INVALID),
             (0, OFF1, INVALID), (8, OFF2, INVALID), (2, 1 << 31, UNSUPPORTED)))
    refused(lib.sg_pack8, [P, 40000, 4, 8, BF, 0, P, 40000, P, None], ((3, 32769, UNSUPPORTED),))
    refused(lib.sg_unpack8, [P, 8, P, 4, 8, 0, P, 8, F32, None],
            ((0, None, INVALID), (2, None, INVALID), (6, None, INVALID), (1, 7, INVALID), (7, 7, INVALID),
             (5, 1, INVALID), (8, E4M3, INVALID), (6, OFF2, INVALID), (2, OFF2, INVALID), (3, -1, INVALID)))
    # no rows: nothing to do, nothing to point at
    assert lib.sg_pack8(None, 8, 0, 8, BF, 128, None, 8, None, None) == 0
    assert lib.sg_unpack8(None, 8, None, 0, 8, 0, None, 8, F32, None) == 0


def test_block_norm_refusals_and_work(lib):
    fwd = [P, 8, P, 8, 4, 8, F16, P, P, P, 1.0, 1e-6, P, 8, P, P, P, 8, P, 8, P, P, 8, P, P, 8, P, None]
    refused(lib.sg_block_norm_fwd, fwd,
            ((0, None, INVALID), (7, None, INVALID), (9, None, INVALID), (20, None, INVALID), (23, None, INVALID),
             (26, None, INVALID), (1, 7, INVALID), (3, 7, INVALID), (13, 7, INVALID), (17, 7, INVALID),
             (19, 7, INVALID), (22, 7, INVALID), (25, 7, INVALID), (6, E4M3, INVALID), (10, float("nan"), INVALID),
             (10, 1e39, INVALID), (11, -1.0, INVALID), (11, float("inf"), INVALID), (14, OFF2, INVALID),
             (15, OFF2, INVALID), (20, OFF2, INVALID), (23, OFF2, INVALID), (26, OFF2, INVALID), (8, OFF1, INVALID),
             (4, -1, INVALID), (5, 0, INVALID)))
    none = list(fwd)
    none[16] = none[18] = None
    assert lib.sg_block_norm_fwd(*none) == INVALID  # neither y nor y8
    wide = list(fwd)
    wide[5] = 16385
    assert lib.sg_block_norm_fwd(*wide) == UNSUPPORTED
    none = list(fwd)
    none[4] = 0
    none[0] = none[16] = None
    assert lib.sg_block_norm_fwd(*none) == 0

    n = C.c_int64(-1)
    assert lib.sg_block_norm_bwd_work(1000, 512, C.byref(n)) == 0 and n.value >= 2 * 512 * 4
    need = n.value
    assert lib.sg_block_norm_bwd_work(1000, 512, None) == INVALID
    assert lib.sg_block_norm_bwd_work(1000, 16385, C.byref(n)) == UNSUPPORTED
    bwd = [P, 512, P, 512, None, P, 512, None, P, 512, 1000, 512, F32, P, P, P, 1.0, P, P, P, 512, P, 512, P, P, P, P,
           need, None]
    refused(lib.sg_block_norm_bwd, bwd,
            ((0, None, INVALID), (2, None, INVALID), (5, None, INVALID), (13, None, INVALID), (15, None, INVALID),
             (17, None, INVALID), (18, None, INVALID), (21, None, INVALID), (26, None, INVALID), (27, need - 1, INVALID),
             (4, P, INVALID), (7, P, INVALID), (14, None, INVALID), (1, 511, INVALID), (3, 511, INVALID),
             (6, 511, INVALID), (9, 511, INVALID), (20, 511, INVALID), (22, 511, INVALID), (26, OFF1, INVALID),
             (17, OFF2, INVALID), (23, OFF2, INVALID), (24, OFF2, INVALID), (25, OFF2, INVALID),
             (16, float("inf"), INVALID), (12, E4M3, INVALID)))
    held = list(bwd)
    held[4], held[7] = P, OFF2
    assert lib.sg_block_norm_bwd(*held) == INVALID
    # with 8-bit rows any address will do for x, not for dy
    held[7], held[0] = P, OFF1
    assert lib.sg_block_norm_bwd(*held) == INVALID and "dy" in sgpkg.last_error()


def test_linear_refusals_and_work(lib):
    n = C.c_int64(-1)

    def work(*a):
        rc = lib.sg_linear8_work(*a, C.byref(n))
        return n.value if rc == 0 else rc

    assert work(P, 64, 300, 64, P, 64, 1000, None, 0, 0) > 0
    assert work(P, 64, 0, 64, P, 64, 1000, None, 0, 0) == 0
    back = work(P, 64, 100, 64, P, 64, 1000, P, 1000, 1)
    # dout's rows that do not start on 16 bytes are copied
    assert work(P, 64, 100, 64, P, 64, 1000, P, 1001, 1) >= back + 100 * 1000 * 2
    assert work(P, 64, 100, 64, P, 64, 1000, OFF2, 1000, 1) >= back + 100 * 1000 * 2
    for bad in ((P, 64, -1, 64, P, 64, 1000, None, 0, 0), (P, 64, 1, 0, P, 64, 1000, None, 0, 0),
                (P, 64, 1, 64, P, 64, 0, None, 0, 0), (P, 63, 1, 64, P, 64, 1000, None, 0, 0),
                (P, 64, 1, 64, P, 63, 1000, None, 0, 0)):
        assert work(*bad) == INVALID, bad
    assert work(P, 64, 1 << 25, 64, P, 64, 1000, None, 0, 0) == UNSUPPORTED
    assert work(P, 64, 1 << 24, 64, P, 64, 1 << 24, None, 0, 0) == UNSUPPORTED
    assert lib.sg_linear8_work(P, 64, 1, 64, P, 64, 1, None, 0, 0, None) == INVALID
    big = 1 << 40
    refused(lib.sg_linear8_fwd, [P, 64, P, 300, 64, P, 64, P, 1000, P, 1000, BF, P, big, P, None],
            ((0, None, INVALID), (2, None, INVALID), (5, None, INVALID), (7, None, INVALID), (9, None, INVALID),
             (12, None, INVALID), (13, 16, INVALID), (12, C.c_void_p(16), INVALID), (10, 999, INVALID),
             (11, E4M3, INVALID), (9, OFF1, INVALID), (2, OFF2, INVALID), (7, OFF2, INVALID), (14, OFF2, INVALID)))
    bwd = [P, 64, P, 0, 4, 64, P, 64, P, 1000, P, 1000, BF, P, 64, P, 64, P, big, P, None]
    refused(lib.sg_linear8_bwd, bwd,
            ((0, None, INVALID), (2, None, INVALID), (6, None, INVALID), (8, None, INVALID), (10, None, INVALID),
             (17, None, INVALID), (18, 16, INVALID), (3, 64, INVALID), (12, F32, INVALID), (11, 999, INVALID),
             (14, 63, INVALID), (16, 63, INVALID), (13, OFF1, INVALID), (15, OFF1, INVALID), (10, OFF1, INVALID),
             (2, OFF2, INVALID), (8, OFF2, INVALID), (19, OFF2, INVALID)))
    neither = list(bwd)
    neither[13] = neither[15] = None
    assert lib.sg_linear8_bwd(*neither) == INVALID
    # no rows: dx alone has nothing to do
    none = [None, 64, None, 0, 0, 64, P, 64, P, 1000, None, 1000, BF, None, 64, None, 64, None, 0, None, None]
    assert lib.sg_linear8_bwd(*none) == 0, sgpkg.last_error()
    assert lib.sg_linear8_status(None, 1) == INVALID


@pytest.mark.parametrize("T,H,N", [(1, 64, 1 << 24), (300, 4096, 262144), (65536, 4096, 16384)])
def test_forward_work_memory_is_bounded(lib, T, H, N):
    """x in 16 bits, at most 256 MB of W in 16 bits, and parts of a split of at
    most four turns of the tiles (a tile of fp32 sums is 256 KB for two CTAs)."""
    n = C.c_int64(-1)
    assert lib.sg_linear8_work(P, H, T, H, P, H, N, None, 0, 0, C.byref(n)) == 0
    assert 0 <= n.value <= (256 << 20) + 2 * T * H + 4 * 152 * 131072 + 4096
