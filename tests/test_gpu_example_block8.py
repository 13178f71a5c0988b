"""The example of a block's end and a linear layer on 8-bit integers runs, its
gradients are the formulas' and its tokens one by one give what the batch
gave."""
import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from oracle import blocks8 as orc

pytestmark = pytest.mark.gpu

PATH = Path(__file__).resolve().parents[1] / "examples" / "block8.py"


@pytest.fixture(scope="module")
def example():
    sg.build()
    spec = importlib.util.spec_from_file_location("block8", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("rows", [6, 256])
def test_runs(example, rows):
    b, losses, served = example.main(["--rows", str(rows), "--features", "256", "--outputs", "300", "--steps", "3"])
    assert all(np.isfinite(losses)) and bool(torch.isfinite(served).all())


def test_gradients_and_single_tokens(example):
    """The gradients from what the step kept, by the formulas in 64 bits.  dW and
    dy take bf16's rounding of a value (2^-8) and of the result once each, dx and
    dresidual that of dy and their own; 2^-6 of the largest element of a result has
    room for both."""
    rows, cols, outs = 40, 256, 300
    b = example.Block(rows, cols, outs, alpha=0.75)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, res, di = (torch.randn((rows, cols), generator=g, device="cuda").bfloat16() for _ in range(3))
    dz = torch.randn((rows, outs), generator=g, device="cuda").bfloat16()
    z = b.forward(x, res).clone()
    b.backward(dz, di)
    dy, dW = orc.linear8_grad(f64(b.y8), f64(b.y_scale), f64(b.W8), f64(b.W_scale), f64(dz))
    u, x8 = orc.values8(f64(b.u8), f64(b.u_scale)), orc.values8(f64(b.x8), f64(b.x_scale))
    want = orc.block_norm_grad(dy, u, x8, f64(b.post), f64(b.gate), f64(b.pre), 0.75, f64(b.rstd_x), f64(b.rstd_u), f64(di))
    for got, w in ((b.dW, dW), (b.dy, dy), (b.dx, want["dx"]), (b.dres, want["dresidual"]), (b.dpost, want["dpost"]),
                   (b.dgate, want["dgate"]), (b.dpre, want["dpre"])):
        assert np.abs(f64(got) - w).max() <= 2.0 ** -6 * np.abs(w).max()
    one = example.Block(1, cols, outs, alpha=0.75)
    one.W8, one.W_scale = b.W8, b.W_scale
    for i in (0, 17, rows - 1):
        # the same integers: the sums are exact in either kernel
        assert torch.equal(one.forward(x[i:i + 1], res[i:i + 1])[0], z[i])


def test_serving_in_the_first_rows_of_the_same_buffers(example):
    """A block over fewer rows has the same weights and buffers, and leaves the rows
    behind its own as they are."""
    b = example.Block(40, 256, 300)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, res = (torch.randn((40, 256), generator=g, device="cuda").bfloat16() for _ in range(2))
    z = b.forward(x, res).clone()
    one = b.first(1)
    assert all(getattr(one, k).data_ptr() == getattr(b, k).data_ptr() for k in ("W", "W8", "W_scale", "z", "y8", "status"))
    for i in (39, 17, 5):
        assert torch.equal(one.forward(x[i:i + 1], res[i:i + 1])[0], z[i])
        assert torch.equal(b.z[0], z[i]) and torch.equal(b.z[1:], z[1:])
    few = b.first(7)
    assert torch.equal(few.forward(x[20:27], res[20:27]), z[20:27]) and torch.equal(b.z[7:], z[7:])
