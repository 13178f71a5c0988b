"""Blocks on 8-bit integers at the ends of what they take."""
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import E, HALF, TYPES, check_forward, check_gradients, rand, rand8, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


# ---------------------------------------------------------------- fp16 gradients of -128
# A scale s times q = -128 passes fp16's largest number where s, times the common
# power of two, is 511.875 or more (65520 rounds to infinity).  check_gradients' bounds
# hold as they are: the largest scale is brought to at least 255.9, so half of fp16's
# smallest step is at most 2^-25 / 255.9 = 1.0005 2^-33 of it for each term, and they
# have 127 2^-39 = 0.99 2^-32.
TOPS = [1 - 2.0 ** -24, 1 - 2.0 ** -12, 1 - 2.0 ** -12 - 2.0 ** -24, 1.0, 1 + 2.0 ** -23]


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("T,H,N,group", [(40, 200, 300, 0), (130, 256, 500, 128), (110, 8200, 64, 128)])
def test_linear_backward_f16_of_the_lowest_integer(T, H, N, group, top):
    x8, W8 = rand8(T, H, 1), rand8(N, H, 2)
    x8[:, ::7] = -128
    W8[:, ::5] = -128
    ws = scales(N, 4)
    xs = scales(T * -(-H // 128), 3).reshape(T, -1) if group else scales(T, 3)
    # the largest of all, next to a power of two
    ws[N // 2] = top * 2.0 ** -5
    xs.view(-1)[T // 2] = top * 2.0 ** -5
    dout = rand(T, N, "f16", 5, std=0.1)
    dx, dW = (torch.empty(s, dtype=torch.float16, device="cuda") for s in ((T, H), (N, H)))
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW)
    check_gradients(x8, xs, W8, ws, dout, dx, dW, "f16")


# ---------------------------------------------------------------- scales of very small and large rows
def scale_rows(rows, cols, size, weight, dtype, pad=0, shift=0):
    """(rms norm's input u of rows as large as `size` says in turn, pre_weight): u
    comes through the residual, with a gate of 0."""
    u = rand(rows, cols, dtype, 2, pad, shift)
    by = torch.tensor([size[i % len(size)] for i in range(rows)], device="cuda", dtype=torch.float64)[:, None]
    u.copy_(u.double() * by)
    pre = (weight * (1 + 0.1 * rand(1, cols, "f32", 3)[0].double())).to(TYPES[dtype])
    return u, pre


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,weight", [((1.0, 1e-15, 1e-17, 0.0, 3.0), 1e-28), ((1e17, 1.0), 1e22), ((0.0, 1.0), 1.0)],
                         ids=["small", "large", "zeros"])
@pytest.mark.parametrize("rows,cols", [(9, 64), (5000, 264), (2500, 768), (7, 1001), (700, 4096), (400, 6000), (200, 9000)])
def test_block_norm_8_bit_scales_where_u_times_its_weight_leaves_fp32(rows, cols, size, weight, dtype, pad, shift):
    """y's scale is by max |y|, of which neither factor nor product has to be an
    fp32 number with all its bits: u pre is not, where u is small or large and pre
    too.  Bounds: as for ordinary rows (a relative 4 E for 160 roundings and the
    division, half a step)."""
    u, pre = scale_rows(rows, cols, size, weight, dtype, pad, shift)
    x, post = rand(rows, cols, dtype, 1, pad, shift), torch.ones(cols, dtype=TYPES[dtype], device="cuda")
    y8, s = torch.empty((rows, cols), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    ru, got = torch.empty(rows, device="cuda"), torch.empty_like(u)
    eps = 1e-38
    sg.sg_block_norm_fwd(x, post, pre, eps, residual=u, gate=torch.zeros_like(post), u=got, rstd_u=ru, y8=y8, y8_scale=s)
    assert torch.equal(got, u)
    u64 = u.double()
    y = u64 * (u64.square().mean(1, keepdim=True) + eps).rsqrt() * pre.double()
    top = y.abs().amax(1)
    assert bool(((s.double() - top / 127).abs() <= 2 * E * top / 127).all())
    assert bool(((y8.double() * s.double()[:, None] - y).abs() <= s.double()[:, None] * (0.5 + 127 * 4 * E)).all())


# ---------------------------------------------------------------- the longest sums, the largest matrices
@pytest.mark.parametrize("T", [1, 5, 100, 600])
def test_linear_of_the_longest_rows(T):
    """2^20 inputs: sums of 1024 parts, each of 1024 terms."""
    H, N = 1 << 20, 300
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    out, status = torch.empty((T, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out, status=status)
    check_forward(x8, xs, W8, ws, out, "f32")
    dout = rand(T, N, "bf16", 5)
    dx, dW = (torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((T, H), (N, H)))
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
    for got, a, b in ((dx, dout.double(), W8.double() * ws.double()[:, None]),
                      (dW, dout.double().t(), x8.double() * xs.double()[:, None])):
        want, terms = a @ b, a.abs() @ b.abs()
        # the values' rounding, the tensor cores' of sums of 1024, parts in fp32
        assert bool(((got.double() - want).abs() <= HALF["bf16"] * want.abs() * 1.001 +
                     (HALF["bf16"] + 2.0 ** -16 + 68 * 2.0 ** -24) * terms).all())
    assert int(status) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,N", [(3, 1 << 24), (1 << 24, 16)])
def test_linear_backward_beyond_2_31_elements(T, N, dtype):
    """As many channels or tokens as there may be: dW or dx has more than 2^31
    elements, and the other one sums over 2^24 terms.  Bounds as test_gpu_blocks8
    has them, those sums in turn of 1024 terms (16384 roundings of 2^-24 in one
    part of K)."""
    H = 136
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    dout = rand(T, N, dtype, 5, std=0.01)
    dx, dW = (torch.full(s, float("nan"), dtype=TYPES[dtype], device="cuda") for s in ((T, H), (N, H)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
    assert int(status) == 0
    at = lambda n: torch.cat([torch.arange(0, min(n, 200)), torch.randint(0, n, (200,)), torch.arange(max(0, n - 200), n)]).cuda()  # noqa: E731
    for got, a, q, s in ((dx, dout, W8, ws), (dW, dout.t(), x8, xs)):
        rows = at(a.shape[0]) if a.shape[0] > 1000 else torch.arange(a.shape[0], device="cuda")
        want, terms, low = (torch.zeros((len(rows), H), dtype=torch.float64, device="cuda") for _ in range(3))
        for k in range(0, a.shape[1], 1 << 20):
            e, v = a[rows][:, k:k + (1 << 20)].double(), q[k:k + (1 << 20)].double() * s[k:k + (1 << 20)].double()[:, None]
            want += e @ v
            terms += e.abs() @ v.abs()
            low += e.abs().sum(1, keepdim=True) * float(s.max()) * 127 * 2.0 ** -39
        bound = HALF[dtype] * want.abs() * 1.001 + 2.0 ** -25 + (HALF[dtype] + 2.0 ** -16 + (16384 + 67) * 2.0 ** -24) * terms + low
        assert bool(((got[rows].double() - want).abs() <= bound).all())
        assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T,H,N", [(1, 130, 77), (40, 300, 500), (130, 200, 300), (600, 520, 1000)])
def test_linear_backward_of_gradients_that_are_not_finite(T, H, N, dtype, shift):
    """They reach their token's dx and their channel's dW alone."""
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    dout = rand(T, N, dtype, 5, -(N + shift) % 8, shift)
    out = []
    for bad in (None, float("nan"), float("inf")):
        if bad is not None:
            dout[T - 1, N - 1] = bad
        dx, dW = (torch.empty(s, dtype=TYPES[dtype], device="cuda") for s in ((T, H), (N, H)))
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW)
        out.append((dx, dW))
    for dx, dW in out[1:]:
        assert not bool(torch.isfinite(dx[T - 1]).any()) and not bool(torch.isfinite(dW[N - 1]).any())
        assert torch.equal(dx[:T - 1], out[0][0][:T - 1]) and torch.equal(dW[:N - 1], out[0][1][:N - 1])
    # a channel's or token's scale reaches all that it is summed into
    dout[T - 1, N - 1] = 1.0
    ws[0], xs[0] = float("nan"), float("nan")
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW)
    assert bool(torch.isnan(dx).all()) and bool(torch.isnan(dW).all())
