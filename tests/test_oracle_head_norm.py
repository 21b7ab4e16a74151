"""Pins of the oracle's head norm: closed forms, and torch's own RMS norm."""
import numpy as np
import torch

from oracle import csa_oracle as O


def test_closed_forms():
    x = np.zeros((1, 2, 4))
    x[0, 1] = [3, 0, 0, 4]
    y = O.head_norm(x, None, 0.75, None)
    assert np.all(y[0, 0] == 0)
    assert np.allclose(y[0, 1], np.array([3, 0, 0, 4]) / np.sqrt(6.25 + 0.75), rtol=1e-15)
    # a quarter turn of the last pair, R = 2: angle = position
    z = O.head_norm(x, np.array([1, 1, 2, 0.5]), 0.75, np.array([1.0]), 2)
    a, b = 0.0, 4 / np.sqrt(7) * 0.5
    assert np.allclose(z[0, 1, 2:], [a * np.cos(1) - b * np.sin(1), a * np.sin(1) + b * np.cos(1)], rtol=1e-14)
    assert np.allclose(z[0, 1, :2], y[0, 1, :2], rtol=0)


def test_agrees_with_torch_and_keeps_the_norm():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 3, 64)) * 10, 1 + 0.1 * rng.standard_normal(64)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-6).numpy()
    flat = O.head_norm(x, w, 1e-6)
    assert np.allclose(flat, want, rtol=1e-13)
    pos = np.array([0, 1, 7, 1 << 20, 33])
    y = O.head_norm(x, w, 1e-6, pos, 16)
    assert np.array_equal(y[..., :48], flat[..., :48]) and np.allclose(y[0], flat[0], rtol=0)
    assert np.allclose((y ** 2).sum(-1), (flat ** 2).sum(-1), rtol=1e-12)
    assert not np.allclose(y[1:, :, 48:], flat[1:, :, 48:], rtol=1e-3)
