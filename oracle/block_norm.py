"""Oracle of the norms before and after a block with its gate and residual scale, and the gradient
(float64).  z = x + alpha a(gate) norm(y) w_post, h = norm(z) w_next, norm(v) = v / sqrt(mean v^2 + eps)."""
from __future__ import annotations

import numpy as np


def _gate(gate, sigmoid):
    """(a, a') as columns or rows that broadcast over [T][H]."""
    if gate is None:
        return np.ones((1, 1)), np.ones((1, 1))
    g = np.asarray(gate, np.float64)
    g = g[:, None] if g.ndim == 1 else g
    if not sigmoid:
        return g, np.ones_like(g)
    a = 0.5 * (1.0 + np.tanh(0.5 * g))
    return a, a * (1.0 - a)


def _inv_rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def block_norm(x, y=None, w_post=None, gate=None, sigmoid=False, alpha=1.0, w_next=None, eps=1e-6):
    """(z, h); z is x without y, h None without w_next."""
    z = x
    if y is not None:
        n = y if w_post is None else y * _inv_rms(y, eps) * w_post
        z = x + alpha * _gate(gate, sigmoid)[0] * n
    return z, None if w_next is None else z * _inv_rms(z, eps) * w_next


def block_norm_bwd(z, dz=None, dh=None, y=None, w_post=None, gate=None, sigmoid=False, alpha=1.0, w_next=None, eps=1e-6):
    """dict of dx, dy, dgate, dw_post, dw_next (those the step has)."""
    H = z.shape[1]
    out = {}
    d = np.zeros_like(z) if dz is None else dz
    if dh is not None:
        r = _inv_rms(z, eps)
        v = w_next * dh
        d = d + r * v - z * r ** 3 * np.sum(z * v, axis=1, keepdims=True) / H
        out["dw_next"] = np.sum(dh * z * r, axis=0)
    out["dx"] = d
    if y is None:
        return out
    a, da = _gate(gate, sigmoid)
    q = _inv_rms(y, eps)
    n = y if w_post is None else y * q * w_post
    if gate is not None:
        g = alpha * da * d * n
        out["dgate"] = g.sum(axis=1) if np.asarray(gate).ndim == 1 else g
    dn = alpha * a * d
    if w_post is None:
        out["dy"] = dn
    else:
        out["dw_post"] = np.sum(dn * y * q, axis=0)
        v = w_post * dn
        out["dy"] = q * v - y * q ** 3 * np.sum(y * v, axis=1, keepdims=True) / H
    return out
