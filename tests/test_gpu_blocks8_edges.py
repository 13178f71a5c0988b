"""Blocks on 8-bit integers at the ends of what they take."""
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import check_gradients, rand, rand8, scales

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
