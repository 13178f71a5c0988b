"""Pins of the 64-bit softmax cross entropy (CPU): torch's own loss, and
differences."""
import numpy as np
import pytest
import torch

from oracle.softmax_ce import softmax_ce


def _case(T=7, H=5, V=13, seed=0):
    r = np.random.RandomState(seed)
    y = r.randint(0, V, T)
    y[::3] = -100
    return r.randn(T, H), r.randn(V, H), y, r.rand(T)


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
def test_against_torch(smoothing):
    h, W, y, c = _case()
    ht, Wt = torch.tensor(h, requires_grad=True), torch.tensor(W, requires_grad=True)
    loss = torch.nn.functional.cross_entropy(ht @ Wt.t(), torch.tensor(y), reduction="none",
                                             label_smoothing=smoothing)
    (loss * torch.tensor(c)).sum().backward()
    got = softmax_ce(h, W, y, c, smoothing=smoothing)
    assert np.allclose(got["loss"], loss.detach().numpy(), atol=1e-12)
    assert np.allclose(got["dh"], ht.grad.numpy(), atol=1e-12)
    assert np.allclose(got["dW"], Wt.grad.numpy(), atol=1e-12)


def test_against_differences():
    h, W, y, c = _case(seed=1)
    r, step = np.random.RandomState(2), 1e-6
    got = softmax_ce(h, W, y, c, smoothing=0.2)
    for k, name in enumerate(("dh", "dW")):
        d = r.randn(*(h, W)[k].shape)
        lo, hi = [h, W], [h, W]
        lo[k], hi[k] = lo[k] - step * d, hi[k] + step * d
        diff = sum(s * (softmax_ce(*a, y, smoothing=0.2)["loss"] * c).sum() for s, a in ((1, hi), (-1, lo)))
        assert abs(diff / (2 * step) - (got[name] * d).sum()) < 1e-7
