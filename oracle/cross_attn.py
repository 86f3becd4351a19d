"""fp64 reference for the softmax blocks' attention to an encoder's states.
TEST INFRASTRUCTURE ONLY.

Per batch row and query head h (key head h // (Hq // Hk)), over the keys the mask
keeps: scores scale q k^T, lse = log sum exp, out = softmax v; a row that keeps no
key has out 0 and lse -inf.  Gradients from the softmax's Jacobian row by row
(dS = P (dP - sum P dP)), in numpy float64; masked keys are left out of every
array rather than set to anything, so their values cannot matter.
"""
from __future__ import annotations

import numpy as np


def forward(q, k, v, mask=None, scale=None):
    """q [B,Tq,Hq,D], k, v [B,S,Hk,D], mask [B,S] or None -> out, lse [B,Hq,Tq]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Tq, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((B, Tq, Hq, D)), np.full((B, Hq, Tq), -np.inf)
    for b, h, p, top, total, keep in _rows(q, k, mask, scale):
        out[b, :, h] = p @ v[b, keep, h // (Hq // k.shape[2])]
        lse[b, h] = (top + np.log(total))[:, 0]
    return out, lse


def backward(q, k, v, d_out, mask=None, scale=None):
    """(dq, dk, dv) of the sum of out * d_out."""
    q, k, v, g = (np.asarray(x, np.float64) for x in (q, k, v, d_out))
    Hq, D = q.shape[2:]
    scale = D ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, h, p, _, _, keep in _rows(q, k, mask, scale):
        hk = h // (Hq // k.shape[2])
        dp = g[b, :, h] @ v[b, keep, hk].T
        ds = scale * p * (dp - np.sum(p * dp, -1, keepdims=True))
        dq[b, :, h] = ds @ k[b, keep, hk]
        dk[b, keep, hk] += ds.T @ q[b, :, h]
        dv[b, keep, hk] += p.T @ g[b, :, h]
    return dq, dk, dv


def _rows(q, k, mask, scale):
    B, _, Hq, _ = q.shape
    S, Hk = k.shape[1], k.shape[2]
    for b in range(B):
        keep = np.arange(S) if mask is None else np.flatnonzero(np.asarray(mask)[b])
        if not len(keep):
            continue
        for h in range(Hq):
            s = scale * (q[b, :, h] @ k[b, keep, h // (Hq // Hk)].T)
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(-1, keepdims=True)
            yield b, h, e / total, top, total, keep
