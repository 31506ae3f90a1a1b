"""CPU oracle of the gated feed-forward block (test infrastructure only), float64.

    G = X Ag + ag,  U = X Au + au,  Y = act(G) * U,  O = R + dropout(Y B + b)
    dZ = dO m / (1-p);  dY = dZ B^T;  dG = dY U act'(G);  dU = dY act(G)
    dX = [dO +] dG Ag^T + dU Au^T;  dA = X^T [dG | dU];  dB = Y^T dZ;  da, db: sums over tokens

A = [Ag | Au] [h, 2 ffn], split over t slices like the MLP block's A (columns of both
halves) and B (rows); act is "silu" (x / (1 + exp(-x))) or "gelu" (the MLP block's tanh
form).  Dropout is the MLP block's.  Each stage is a function of its own, so that a
test can feed it the stored tensors of the stage before.

Pinned by tests/test_oracle_glu.py against autograd in float64, slice invariance and
central differences.
"""
from __future__ import annotations

import numpy as np

from .mlp_oracle import dropout_keep, dropout_scale


def act(x, kind):
    if kind == "silu":
        return x / (1.0 + np.exp(-x))
    return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x**3)))


def act_prime(x, kind):
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    k = np.sqrt(2.0 / np.pi)
    t = np.tanh(k * (x + 0.044715 * x**3))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * x * x)


def gates(X, A, a, t=1):
    """GU [tokens, 2 ffn], slice by slice."""
    ffn = A.shape[1] // 2
    f = ffn // t
    GU = np.empty((X.shape[0], 2 * ffn))
    for half in range(2):
        for i in range(t):
            c = slice(half * ffn + i * f, half * ffn + (i + 1) * f)
            GU[:, c] = X @ A[:, c] + (0.0 if a is None else a[c])
    return GU


def gated(GU, kind):
    ffn = GU.shape[1] // 2
    return act(GU[:, :ffn], kind) * GU[:, ffn:]


def out(Y, B, b, R, p, seed, token_offset=0, t=1):
    f = B.shape[0] // t
    Z = sum(Y[:, i * f:(i + 1) * f] @ B[i * f:(i + 1) * f] for i in range(t))
    if b is not None:
        Z = Z + b
    keep = dropout_keep(Z.shape[0], Z.shape[1], p, seed, token_offset)
    return R + np.where(keep, Z * dropout_scale(p), 0.0)


def d_out(dO, p, seed, token_offset=0):
    """dZ."""
    keep = dropout_keep(dO.shape[0], dO.shape[1], p, seed, token_offset)
    return np.where(keep, dO * dropout_scale(p), 0.0)


def d_gates(dZ, B, GU, kind):
    """dGU."""
    ffn = B.shape[0]
    G, U = GU[:, :ffn], GU[:, ffn:]
    dY = dZ @ B.T
    return np.concatenate([dY * U * act_prime(G, kind), dY * act(G, kind)], axis=1)


def d_input(dGU, A, dO=None):
    return dGU @ A.T + (0.0 if dO is None else dO)


def d_weights(X, dZ, Y, dGU):
    """dA, da, dB, db."""
    return X.T @ dGU, dGU.sum(axis=0), Y.T @ dZ, dZ.sum(axis=0)
