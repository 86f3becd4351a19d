"""Pins of the fp64 oracle of the attention to encoder states (CPU): closed forms,
shared heads, masks, PyTorch's own attention, gradients against autograd and
differences."""
import numpy as np
import pytest
import torch

from oracle import cross_attn as ca
from oracle import sink_window_attn as swa


def draw(B=2, Tq=5, S=7, Hk=2, G=3, D=16, seed=1):
    rng = np.random.default_rng(seed)
    q, g = rng.standard_normal((2, B, Tq, Hk * G, D))
    k, v = rng.standard_normal((2, B, S, Hk, D))
    mask = rng.random((B, S)) < 0.6
    mask[:, 0] = True
    return q, k, v, g, mask


def test_closed_forms():
    q, k, v, _, mask = draw()
    out, lse = ca.forward(0 * q, k, v, mask)
    for b in range(2):
        n = mask[b].sum()
        np.testing.assert_allclose(lse[b], np.log(n))
        np.testing.assert_allclose(out[b, 0, 4], v[b, mask[b], 1].mean(0))
    one = np.zeros_like(mask)
    one[:, 3] = True
    out, lse = ca.forward(q, k, v, one)
    np.testing.assert_allclose(out[1, 2, 0], v[1, 3, 0])
    np.testing.assert_allclose(lse[1, 5, 2], q[1, 2, 5] @ k[1, 3, 1] / 4.0)
    none = np.zeros_like(mask)
    out, lse = ca.forward(q, k, v, none)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_agrees_with_the_streaming_attention_oracle():
    q, k, v, _, _ = draw(Hk=1, G=1)
    out, _ = ca.forward(q, k, v)
    np.testing.assert_allclose(out[0, :, 0], swa.attend(q[0, :, 0], k[0, :, 0], v[0, :, 0]), atol=1e-13)


def test_masked_values_do_not_matter():
    q, k, v, g, mask = draw()
    k2, v2 = k.copy(), v.copy()
    k2[~mask], v2[~mask] = np.nan, np.inf
    for a, b in zip(ca.forward(q, k, v, mask), ca.forward(q, k2, v2, mask)):
        np.testing.assert_array_equal(a, b)
    for a, b in zip(ca.backward(q, k, v, g, mask), ca.backward(q, k2, v2, g, mask)):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("masked", [False, True])
def test_gradients_match_autograd_and_differences(masked):
    q, k, v, g, mask = draw()
    m = mask if masked else None
    dq, dk, dv = ca.backward(q, k, v, g, m)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    kk, vv = (x.repeat_interleave(3, 2) for x in t[1:])
    s = torch.einsum("bthd,bshd->bhts", t[0], kk) / 4.0
    if masked:
        s = s.masked_fill(~torch.tensor(mask)[:, None, None], -np.inf)
    out = torch.einsum("bhts,bshd->bthd", s.softmax(-1), vv)
    np.testing.assert_allclose(ca.forward(q, k, v, m)[0], out.detach().numpy(), atol=1e-13)
    out.backward(torch.tensor(g))
    for a, b in zip((dq, dk, dv), t):
        np.testing.assert_allclose(a, b.grad.numpy(), atol=1e-12)
    rng = np.random.default_rng(2)
    for x, d in ((q, dq), (k, dk), (v, dv)):
        step = rng.standard_normal(x.shape)
        f = lambda e: np.sum(g * ca.forward(*(y + e * step if y is x else y for y in (q, k, v)), m)[0])  # noqa: E731
        assert (f(1e-5) - f(-1e-5)) / 2e-5 == pytest.approx(np.sum(step * d), rel=1e-6)
