"""Pins of the fp64 norm / rotary oracle (CPU): hand values, invariances, and its
gradients against differences and against autograd of the definition."""
import numpy as np
import pytest
import torch

from oracle import norm_rope as nr


def test_rotation_by_hand():
    x = np.zeros((1, 1, 1, 16))
    x[..., 0], x[..., 1] = 3.0, 4.0
    ang = np.zeros((1, 1, 8))
    ang[..., 0] = np.pi / 2
    out = nr.turn(x, ang, "interleaved", amplitude=2.0)
    np.testing.assert_allclose(out[0, 0, 0, :2], [-8.0, 6.0], atol=1e-14)
    x = np.zeros((1, 1, 1, 16))
    x[..., 0], x[..., 8] = 3.0, 4.0
    out = nr.turn(x, ang, "half")
    np.testing.assert_allclose(out[0, 0, 0, [0, 8]], [-4.0, 3.0], atol=1e-14)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scores_depend_on_distance_only(layout):
    rng = np.random.default_rng(3)
    f = 10000.0 ** (-np.arange(8) / 8)
    q, k = rng.standard_normal((2, 1, 1, 1, 32))

    def score(m, n):
        at = lambda p: nr.angles(np.full((1, 1, 1), p), f, (8,))  # noqa: E731
        return np.sum(nr.turn(q, at(m), layout) * nr.turn(k, at(n), layout))
    assert score(7, 3) == pytest.approx(score(1007, 1003), abs=1e-9)
    assert abs(score(7, 3) - score(7, 4)) > 1e-3


def test_norm_is_scale_free_and_unit():
    x = np.random.default_rng(4).standard_normal((2, 3, 2, 48))
    y = nr.norm(x, None, 0.0)
    np.testing.assert_allclose(np.mean(y * y, -1), 1.0, atol=1e-13)
    np.testing.assert_allclose(nr.norm(7.0 * x, None, 0.0), y, atol=1e-13)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients_match_autograd_and_differences(layout):
    rng = np.random.default_rng(5)
    B, T, H, D, R = 2, 3, 2, 32, 16
    x, dy = rng.standard_normal((2, B, T, H, D))
    w = 1.0 + 0.3 * rng.standard_normal(D)
    ang = nr.angles(rng.integers(0, 50, (B, T, 2)), 100.0 ** (-np.arange(8) / 8), (5, 3))
    dx, dw = nr.norm_turn_backward(x, w, 1e-3, dy, ang, layout, 1.3)

    def loss(x, w):
        return np.sum(dy * nr.norm_turn(x, w, 1e-3, ang, layout, 1.3))
    for _ in range(12):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = 1e-5
        assert (loss(x + e, w) - loss(x - e, w)) / 2e-5 == pytest.approx(dx[i], rel=1e-6, abs=1e-8)
        f = np.zeros_like(w)
        f[i[-1]] = 1e-5
        assert (loss(x, w + f) - loss(x, w - f)) / 2e-5 == pytest.approx(dw[i[-1]], rel=1e-6, abs=1e-8)
    a, b = nr.pair_indices(R, layout)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = tx * tw / torch.sqrt((tx * tx).mean(-1, keepdim=True) + 1e-3)
    c, s = (torch.tensor(1.3 * f(ang))[:, :, None] for f in (np.cos, np.sin))
    z = y.clone()
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    z.backward(torch.tensor(dy))
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
