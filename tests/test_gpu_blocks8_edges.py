"""Blocks on 8-bit integers at the ends of what they take."""
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import E, TYPES, check_gradients, rand, rand8, scales

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
