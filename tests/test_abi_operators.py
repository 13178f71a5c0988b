"""CPU-only checks of the operators around the layer: bad arguments are refused
before anything is launched, and work sizes need no GPU."""
import ctypes as C

import pytest

import extreme_label_sparse_gb300 as sgpkg

P = C.c_void_p(256)  # never dereferenced: validation fails first
INVALID, UNSUPPORTED = sgpkg.SG_ERR_INVALID, sgpkg.SG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    sgpkg.build()
    return sgpkg.load()


def test_dropout_refusals(lib):
    ok = [P, 8, 4, 8, sgpkg.SG_BF16, 0.5, 1, 2, P, 8, None]
    for at, bad, want in ((0, None, INVALID), (8, None, INVALID), (1, 7, INVALID), (9, 7, INVALID), (2, -1, INVALID),
                          (3, 0, INVALID), (4, 3, INVALID), (4, 9, INVALID), (5, 1.5, INVALID),
                          (5, float("nan"), INVALID), (0, C.c_void_p(257), INVALID), (2, 1 << 31, UNSUPPORTED)):
        args = list(ok)
        args[at] = bad
        assert lib.sg_dropout(*args) == want, (at, bad, sgpkg.last_error())
        assert "sg_dropout" in sgpkg.last_error()


def test_norm_refusals_and_work(lib):
    ok = [P, 8, None, 8, 4, 8, sgpkg.SG_F16, P, 1e-6, 0.0, 1, 2, None, 8, None, P, 8, None, 8, None, None]
    for at, bad, want in ((0, None, INVALID), (7, None, INVALID), (15, None, INVALID), (17, P, INVALID),
                          (8, -1.0, INVALID), (8, float("inf"), INVALID), (9, 2.0, INVALID), (1, 4, INVALID),
                          (5, 40000, UNSUPPORTED)):
        args = list(ok)
        args[at] = bad
        assert lib.sg_add_rmsnorm_fwd(*args) == want, (at, bad, sgpkg.last_error())
    n = C.c_int64(-1)
    assert lib.sg_add_rmsnorm_bwd_work(1000, 512, C.byref(n)) == 0 and n.value > 0
    assert lib.sg_add_rmsnorm_bwd_work(1000, 512, None) == INVALID
    bwd = [P, 8, P, 8, None, 8, 4, 8, sgpkg.SG_F32, P, P, 0.0, 1, 2, P, 8, None, 8, P, P, 1 << 30, None]
    for at, bad, want in ((0, None, INVALID), (2, None, INVALID), (10, None, INVALID), (14, None, INVALID),
                          (19, None, INVALID), (20, 8, INVALID), (15, 4, INVALID), (7, 32769, INVALID)):
        args = list(bwd)
        args[at] = bad
        if at == 7:
            args[1] = args[3] = args[5] = args[15] = args[17] = 40000
            want = UNSUPPORTED
        assert lib.sg_add_rmsnorm_bwd(*args) == want, (at, bad, sgpkg.last_error())


def test_softmax_refusals_and_work(lib):
    n = C.c_int64(-1)

    def work(h, ldh, T, H, W, ldw, V, dtype, backward):
        rc = lib.sg_softmax_ce_work(h, ldh, T, H, W, ldw, V, dtype, backward, C.byref(n))
        return n.value if rc == 0 else rc

    bf = sgpkg.SG_BF16
    aligned = work(P, 64, 100, 64, P, 64, 1000, bf, 1)
    assert aligned > 0 and work(P, 64, 0, 64, P, 64, 1000, bf, 1) == 0
    # rows that do not start on 16 bytes are copied: room for W, and for h
    assert work(P, 64, 100, 64, P, 65, 1000, bf, 1) >= aligned + 1000 * 64 * 2
    assert work(P, 64, 100, 64, C.c_void_p(258), 64, 1000, bf, 1) >= aligned + 1000 * 64 * 2
    assert work(P, 61, 100, 60, P, 64, 1000, bf, 1) >= work(P, 64, 100, 60, P, 64, 1000, bf, 1) + 100 * 60 * 2
    for bad in ((P, 64, -1, 64, P, 64, 1000, bf, 0), (P, 64, 1, 0, P, 64, 1000, bf, 0), (P, 64, 1, 64, P, 64, 0, bf, 0),
                (P, 63, 1, 64, P, 64, 1000, bf, 0), (P, 64, 1, 64, P, 63, 1000, bf, 0),
                (P, 64, 1, 64, P, 64, 1000, sgpkg.SG_F32, 0), (P, 64, 1, 64, P, 64, 1000, sgpkg.SG_E4M3, 1)):
        assert work(*bad) == INVALID, bad
    assert work(P, 64, 1 << 25, 64, P, 64, 1000, bf, 0) == UNSUPPORTED
    fwd = [P, 64, None, 4, 64, P, 64, None, 1000, bf, P, -100, 0.0, P, P, P, 1 << 40, None, None]
    for at, bad in ((0, None), (5, None), (10, None), (13, None), (14, None), (15, None), (16, 16), (2, P), (7, P),
                    (12, -0.5), (12, 1.5), (15, C.c_void_p(16))):
        args = list(fwd)
        args[at] = bad
        assert lib.sg_softmax_ce_fwd(*args) == INVALID, (at, bad, sgpkg.last_error())
    bwd = [P, 64, 4, 64, P, 64, 1000, bf, P, -100, 0.0, P, P, P, 64, P, 64, P, 1 << 40, None, None]
    for at, bad in ((0, None), (4, None), (8, None), (11, None), (12, None), (14, 63), (16, 63), (17, None), (18, 16),
                    (13, C.c_void_p(257))):
        args = list(bwd)
        args[at] = bad
        assert lib.sg_softmax_ce_bwd(*args) == INVALID, (at, bad, sgpkg.last_error())
    args = list(bwd)
    args[13] = args[15] = None
    assert lib.sg_softmax_ce_bwd(*args) == INVALID


def test_softmax_backward_of_no_rows_with_dh_alone(lib):
    """No rows: dh has no elements, so its pointer may be NULL, and without dW
    there is nothing to do."""
    args = [None, 64, 0, 64, P, 64, 1000, sgpkg.SG_BF16, None, -100, 0.0, None, None, None, 64, None, 64, None, 0, None,
            None]
    assert lib.sg_softmax_ce_bwd(*args) == 0, sgpkg.last_error()
    args[2] = 1
    assert lib.sg_softmax_ce_bwd(*args) == INVALID


def test_vectors_off_their_elements_are_refused(lib):
    """Each fp32 or int32 vector by itself, two bytes off its elements."""
    off, bf = C.c_void_p(258), sgpkg.SG_BF16
    calls = (
        (lib.sg_add_rmsnorm_fwd, [P, 8, None, 8, 4, 8, bf, P, 1e-6, 0.0, 1, 2, None, 8, P, P, 8, P, 8, P, None],
         (14, 19)),
        (lib.sg_add_rmsnorm_bwd, [P, 8, P, 8, None, 8, 4, 8, bf, P, P, 0.0, 1, 2, P, 8, None, 8, P, P, 1 << 30, None],
         (10, 18, 19)),
        (lib.sg_softmax_ce_fwd, [P, 64, P, 4, 64, P, 64, P, 1000, sgpkg.SG_E4M3, P, -100, 0.0, P, P, P, 1 << 40, P, None],
         (2, 7, 10, 13, 14, 17)),
        (lib.sg_softmax_ce_bwd, [P, 64, 4, 64, P, 64, 1000, bf, P, -100, 0.0, P, P, P, 64, P, 64, P, 1 << 40, P, None],
         (8, 11, 12, 19)),
    )
    for call, ok, places in calls:
        for at in places:
            args = list(ok)
            args[at] = off
            assert call(*args) == INVALID, (call.__name__, at, sgpkg.last_error())
            assert "align" in sgpkg.last_error()


@pytest.mark.parametrize("T,H,V", [(1, 64, 1 << 30), (300, 64, 1 << 30), (8192, 512, 262144), (65536, 512, 262144),
                                   (1 << 20, 64, 1 << 20), (1 << 24, 64, 1 << 20), (1 << 24, 64, 100)])
def test_forward_work_memory_is_bounded(lib, T, H, V):
    """Partial results of at most 256 MB, and 4 to 16 bytes a row (rows here
    start on 16 bytes, so nothing is copied)."""
    n = C.c_int64(-1)
    assert lib.sg_softmax_ce_work(P, H, T, H, P, H, V, sgpkg.SG_BF16, 0, C.byref(n)) == 0
    assert 0 < n.value <= (256 << 20) + 16 * T + 4096


def test_softmax_status_wants_a_place(lib):
    assert lib.sg_softmax_ce_status(None, 1) == INVALID
