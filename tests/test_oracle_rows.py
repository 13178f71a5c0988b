"""Pins of the 64-bit restatements of dropout and RMS norm (CPU)."""
import numpy as np
import pytest

from oracle import rows as orc


def test_philox_known_answers():
    """The published known-answer vectors of Philox4x32-10."""
    ones = 0xFFFFFFFF
    assert orc.philox4x32([0, 0, 0, 0], [0, 0]) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert orc.philox4x32([ones] * 4, [ones] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert orc.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_follows_the_counter_layout():
    seed, offset, p = 0x0123456789ABCDEF, 0xFEDCBA9876543210, 0.3
    keep = orc.dropout_keep(5, 21, p, seed, offset)
    for r in range(5):
        for c in range(21):
            words = orc.philox4x32([c // 8, r, offset & 0xFFFFFFFF, offset >> 32], [seed & 0xFFFFFFFF, seed >> 32])
            bits = (words[c % 8 // 2] >> (16 * (c % 2))) & 0xFFFF
            assert keep[r, c] == (bits >= round(p * 65536))


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_share_kept(p):
    n = 512 * 1000
    got = orc.dropout_keep(512, 1000, p, 7, 11).mean()
    assert abs(got - (1 - p)) < 5 * np.sqrt(max(p * (1 - p), 1e-12) / n) + 2.0 ** -16


def test_norm_gradient_against_differences():
    r = np.random.RandomState(0)
    u, w, dy = r.randn(6, 19), r.randn(19), r.randn(6, 19)
    d, dv, step = r.randn(6, 19), r.randn(19), 1e-5
    y, rstd = orc.add_rmsnorm(u, w, 1e-3)
    assert np.allclose(y, u / np.sqrt((u ** 2).mean(1, keepdims=True) + 1e-3) * w)
    du, dw = orc.add_rmsnorm_grad(dy, u, w, rstd)

    def loss(uu, ww):
        return (orc.add_rmsnorm(uu, ww, 1e-3)[0] * dy).sum()

    assert abs((du * d).sum() - (loss(u + step * d, w) - loss(u - step * d, w)) / (2 * step)) < 1e-7
    assert abs((dw * dv).sum() - (loss(u, w + step * dv) - loss(u, w - step * dv)) / (2 * step)) < 1e-7
