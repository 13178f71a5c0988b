"""The example that runs dropout, RMS norm, both heads and 8-bit scoring
together: its losses fall, and its 8-bit scores are close to 16-bit ones."""
import importlib.util
from pathlib import Path

import pytest
import torch

import extreme_label_sparse_gb300 as sg

pytestmark = pytest.mark.gpu

PATH = Path(__file__).resolve().parents[1] / "examples" / "softmax_head.py"


@pytest.fixture(scope="module")
def example():
    sg.build()
    spec = importlib.util.spec_from_file_location("softmax_head", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("rows", [96, 256])
def test_losses_fall(example, rows):
    history, scored = example.main(["--rows", str(rows), "--features", "128", "--head", "1000", "--tail", "2048",
                                    "--steps", "25"])
    assert history[-1][0] < 0.8 * history[0][0] and history[-1][1] < history[0][1]
    assert bool(torch.isfinite(scored).all())


def test_8_bit_scores_are_close_to_16_bit_ones(example):
    """Rounding to e4m3 moves an element by at most 2^-4 of it: a logit, a sum of
    H products of independent signs, by about sqrt(2) 2^-4 / sqrt(3) of its
    terms' root mean square, some 0.05 here; 0.5 is ten times that."""
    m = example.Model(64, 256, 2000, 2048)
    x, res = (torch.randn((64, 256), device="cuda").bfloat16() for _ in range(2))
    y = torch.randint(0, 2000, (64,), device="cuda", dtype=torch.int32)
    h, loss, lse = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    sg.sg_add_rmsnorm_fwd(x, m.weight, example.EPS, residual=res, y=h)
    sg.sg_softmax_ce_fwd(h, m.W, y, loss, lse)
    assert float((m.score(x, res, y) - loss).abs().max()) < 0.5
    m.layout.close()
