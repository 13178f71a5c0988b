"""Pins of the 64-bit restatements of 8-bit rows, the norms around a block and
the linear layer on 8-bit integers (CPU)."""
import numpy as np
import pytest

from oracle import blocks8 as orc


def test_pack_by_hand():
    x = np.array([[127.0, -63.5, 0.4, 0.5, 1.5, -0.0], [0, 0, 0, 0, 0, 0], [1, 2, np.inf, 0, 0, 0]], dtype=np.float32)
    q, s = orc.pack8(x, 0)
    assert q.tolist() == [[127, -64, 0, 0, 2, 0], [0] * 6, [0] * 6]  # ties to even
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2])


@pytest.mark.parametrize("cols", [1, 128, 129, 300])
@pytest.mark.parametrize("group", [0, 128])
def test_values_are_within_half_a_step(cols, group):
    x = np.random.RandomState(cols).randn(7, cols).astype(np.float32) * 1e3
    q, s = orc.pack8(x, group)
    assert s.shape == ((7, -(-cols // 128)) if group else (7,))
    step = orc.values8(np.ones_like(q), s)
    # half a step, and fp32's rounding of x (127 (1 / a)) of up to 127
    assert (np.abs(orc.values8(q, s) - x) <= step * (0.5 + 127 * 2.0 ** -22)).all()
    assert np.abs(q).max() == 127


def test_block_norm_gradient_against_differences():
    r = np.random.RandomState(0)
    x, res, dy, du_in = (r.randn(5, 19) for _ in range(4))
    post, gate, pre = (1 + 0.3 * r.randn(19) for _ in range(3))
    alpha, eps, step = 1.25, 1e-3, 1e-6

    def loss(x, res, post, gate, pre):
        u, _ = orc.block_norm_u(x, res, post, gate, alpha, eps)
        y = u * orc.rms(u, eps)[:, None] * pre
        return (y * dy).sum() + (u * du_in).sum()

    u, rx = orc.block_norm_u(x, res, post, gate, alpha, eps)
    assert np.allclose(u, alpha * res + gate * (x / np.sqrt((x ** 2).mean(1, keepdims=True) + eps) * post))
    got = orc.block_norm_grad(dy, u, x, post, gate, pre, alpha, rx, orc.rms(u, eps), du_in)
    args = [x, res, post, gate, pre]
    for i, name in enumerate(("dx", "dresidual", "dpost", "dgate", "dpre")):
        d = r.randn(*args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        want = (loss(*up) - loss(*down)) / (2 * step)
        assert abs((got[name] * d).sum() - want) < 1e-6 * (1 + abs(want)), name


def test_linear_gradient_against_differences():
    """The gradients of x = xs x8 and W = ws W8 as real numbers."""
    r = np.random.RandomState(1)
    x8, W8 = r.randint(-128, 128, (4, 300)), r.randint(-128, 128, (6, 300))
    xs, ws, dout = r.rand(4, 3) / 100, r.rand(6) / 100, r.randn(4, 6)
    dx, dW = orc.linear8_grad(x8, xs, W8, ws, dout)
    x, W = orc.values8(x8, xs), orc.values8(W8, ws)
    assert x[1, 130] == x8[1, 130] * xs[1, 1]
    ex, eW = r.randn(*x.shape), r.randn(*W.shape)
    for t in (1e-5,):
        want = ((((x + t * ex) @ W.T) - ((x - t * ex) @ W.T)) * dout).sum() / (2 * t)
        assert abs((dx * ex).sum() - want) < 1e-6 * (1 + abs(want))
        want = (((x @ (W + t * eW).T) - (x @ (W - t * eW).T)) * dout).sum() / (2 * t)
        assert abs((dW * eW).sum() - want) < 1e-6 * (1 + abs(want))
    row = orc.linear8(x8, xs[:, 0], W8, ws)
    assert np.isclose(row[2, 3], xs[2, 0] * ws[3] * int((x8[2].astype(np.int64) * W8[3]).sum()))
