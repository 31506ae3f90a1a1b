"""CPU oracle of the head norms with position rotation (test infrastructure only), float64.

A pair of elements is one complex number and the rotation its product with
exp(i angle); the norm is x / sqrt(mean(x^2) + eps) * w.  Angles are the exact product
of the integer position and the fp32 frequency, in float64.

Pinned by tests/test_oracle_qk_rope.py: norms and inner products that depend on the
difference of two positions only, autograd in float64, central differences.
"""
from __future__ import annotations

import numpy as np


def angles(pos, inv_freq, sections):
    """[tokens, rot / 2] from pos [axes, tokens] and inv_freq [rot / 2]."""
    axis = np.repeat(np.arange(len(sections)), sections)
    return np.asarray(pos, dtype=np.float64)[axis].T * np.asarray(inv_freq, dtype=np.float64)


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, ang, rot, interleaved):
    """x [tokens, heads, d] with its pairs turned by ang [tokens, rot / 2]."""
    i, j = _pairs(rot, interleaved)
    z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * ang)[:, None, :]
    y = x.copy()
    y[..., i], y[..., j] = z.real, z.imag
    return y


def rstd(x, eps):
    return 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)


def fwd(x, w, ang, rot, interleaved, eps):
    n = x if w is None else x * rstd(x, eps) * w
    return turn(n, ang, rot, interleaved)


def bwd(x, w, dy, ang, rot, interleaved, eps):
    """dx, dw (None without the norm)."""
    g = turn(dy, -ang, rot, interleaved)
    if w is None:
        return g, None
    r = rstd(x, eps)
    dw = (g * x * r).sum(axis=(0, 1))
    wg = w * g
    return r * wg - x * r**3 * (wg * x).mean(axis=-1, keepdims=True), dw
