"""Blocks on 8-bit integers at sizes where a CTA has much to do: several units of
both products of the linear layer's backward pass.  Everything is compared, with 64-bit results worked out on the GPU."""
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import HALF, LEAST, TYPES, rand, rand8, scales
from test_linear8_turns import PATHS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def near(got, want, dtype, slack, what):
    """As test_gpu_blocks8.close, on the GPU."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    err = (got - want).abs() - (HALF[dtype] * want.abs() * 1.001 + LEAST[dtype] + slack)
    assert float(err.max()) <= 0, (what, float(err.max()), divmod(int(err.argmax()), got.shape[-1]))


def values(q, scale):
    s = scale.double()
    return q.double() * (s[:, None] if s.dim() == 1 else s.repeat_interleave(128, 1)[:, :q.shape[1]])


# ---------------------------------------------------------------- linear layer
@pytest.mark.parametrize("dtype,group", [("bf16", 128), ("f16", 0)])
@pytest.mark.parametrize("T,H,N", [p[:3] for p in PATHS])
def test_linear_backward_of_several_units_to_a_cluster(T, H, N, dtype, group):
    """Bounds of single elements: those of test_gpu_blocks8 (the values' rounding,
    HALF of each term, 2^-16 for sums of 1024 terms in the tensor cores, fp32 sums of
    parts; fp16's smallest step).

    Of the root mean square: a rounding is off by an even spread of up to half a
    step, HALF / sqrt(3) of the bottom of the value's binade, and so by no more than
    that of the value.  Errors of independent terms add up as their squares do,
    so those of the values are HALF / sqrt(3) of the result, and its own as much
    again: sqrt(2 / 3) HALF = 0.817 HALF where there are many terms, whatever the
    values."""
    x8, W8, ws = rand8(T, H, 1, (-H) % 16), rand8(N, H, 2, (-H) % 16), scales(N, 4)
    xs = scales(T * -(-H // 128), 3).reshape(T, -1) if group else scales(T, 3)
    dout = rand(T, N, dtype, 5, (-N) % 8, std=0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        dx, dW = (torch.full(s, float("nan"), dtype=TYPES[dtype], device="cuda") for s in ((T, H), (N, H)))
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
        got.append((dx, dW))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and int(status) == 0
    d = dout.double()
    for out, a, b, top, what in ((dx, d, values(W8, ws), ws, "dx"), (dW, d.t(), values(x8, xs), xs, "dW")):
        want, terms = a @ b, a.abs() @ b.abs()
        parts = (a.shape[1] / 1024 + 67) * 2.0 ** -24
        low = a.abs().sum(1, keepdim=True) * float(top.max()) * 127 * 2.0 ** -39 if dtype == "f16" else 0.0
        near(out, want, dtype, (HALF[dtype] + 2.0 ** -16 + parts) * terms + low, what)
        if a.shape[1] >= 64:
            rel = float((out.double() - want).norm() / want.norm())
            assert rel <= 0.82 * HALF[dtype], (what, rel / HALF[dtype])
