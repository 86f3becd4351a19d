"""fp64 reference for the softmax blocks' query/key norm and rotary positions.
TEST INFRASTRUCTURE ONLY.

RMS norm of every head row (x weight / sqrt(mean x^2 + eps)) and the rotation of
its first R features by position times frequency, pair i being features i and
i + R/2 ("half") or 2i and 2i + 1 ("interleaved"), and the gradients of both,
in numpy float64 straight from the formulas.  The gradient is written out as
the row's Jacobian (a matrix), not in the folded form the kernels use.
"""
from __future__ import annotations

import numpy as np


def pair_indices(R, layout):
    i = np.arange(R // 2)
    return (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)


def angles(positions, inv_freq, sections):
    """positions [B, T, axes], inv_freq [R/2] -> [B, T, R/2] radians."""
    axis = np.repeat(np.arange(len(sections)), sections)
    return np.asarray(positions, np.float64)[..., axis] * np.asarray(inv_freq, np.float64)


def turn(x, angle, layout, amplitude=1.0, inverse=False):
    """x [B, T, H, D], angle [B, T, R/2]."""
    out = np.array(x, np.float64)
    a, b = pair_indices(2 * angle.shape[-1], layout)
    c = amplitude * np.cos(angle)[:, :, None]
    s = amplitude * np.sin(angle)[:, :, None] * (-1.0 if inverse else 1.0)
    xa, xb = np.asarray(x, np.float64)[..., a], np.asarray(x, np.float64)[..., b]
    out[..., a], out[..., b] = xa * c - xb * s, xa * s + xb * c
    return out


def norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, np.float64)


def norm_turn(x, weight, eps, angle=None, layout="half", amplitude=1.0):
    y = norm(x, weight, eps)
    return y if angle is None else turn(y, angle, layout, amplitude)


def norm_turn_backward(x, weight, eps, dy, angle=None, layout="half", amplitude=1.0):
    """(dx, dweight): per row, y_f = w_f x_f r with r = (mean x^2 + eps)^(-1/2)
    has d y_f / d x_e = w_f (r [f = e] - x_f x_e r^3 / D)."""
    x = np.asarray(x, np.float64)
    g = np.asarray(dy, np.float64)
    if angle is not None:
        g = turn(g, angle, layout, amplitude, inverse=True)
    D = x.shape[-1]
    w = np.ones(D) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1) + eps)
    gw = g * w
    dx = r[..., None] * gw - x * (np.einsum("bthf,bthf->bth", gw, x) * r ** 3 / D)[..., None]
    return dx, np.einsum("bthf,bthf,bth->f", g, x, r)
