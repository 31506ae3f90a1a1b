"""CPU oracle of the attention block with head norms and rotation (test infrastructure
only), float64: the attention block of attn_oracle with qk_rope_oracle's norm and rotation
of its queries and keys between the projection and the core.  ``mirror`` rounds to bf16
where the GPU stores bf16: QKV, QKr, P, O, out, and dZ, dO, dS, the core's dQKV, dQKV, dX.

Pinned by tests/test_oracle_attn_rope.py: angles of zero without the norm give
attn_oracle's block; autograd in float64.
"""
from __future__ import annotations

import math

import numpy as np

from . import qk_rope_oracle as qro
from .mlp_oracle import dropout_keep, dropout_scale, round_bf16


def _rb(x, mirror):
    return round_bf16(x) if mirror else x


def _heads(x, nh):
    return x.reshape(x.shape[0], nh, -1)


def fwd(X, Wqkv, bqkv, Wo, bo, nh, seq_len, p, seed, rope, token_offset=0, mirror=False):
    """rope: dict(wq, wk, ang [tokens, rot/2], rot, inter, eps)."""
    T, h = X.shape
    d = h // nh
    QKV = _rb(X @ Wqkv + bqkv, mirror)
    turned = [_rb(qro.fwd(_heads(QKV[:, k * h:(k + 1) * h], nh), w, rope["ang"], rope["rot"], rope["inter"], rope["eps"]), mirror)
              for k, w in ((0, rope["wq"]), (1, rope["wk"]))]
    V = _heads(QKV[:, 2 * h:], nh)
    P = np.zeros((T // seq_len, nh, seq_len, seq_len))
    O = np.empty((T, nh, d))
    causal = np.tril(np.ones((seq_len, seq_len), dtype=bool))
    for s in range(T // seq_len):
        r = slice(s * seq_len, (s + 1) * seq_len)
        for j in range(nh):
            sc = np.where(causal, turned[0][r, j] @ turned[1][r, j].T / math.sqrt(d), -np.inf)
            e = np.exp(sc - sc.max(axis=1, keepdims=True))
            P[s, j] = _rb(e / e.sum(axis=1, keepdims=True), mirror)
            O[r, j] = P[s, j] @ V[r, j]
    O = _rb(O.reshape(T, h), mirror)
    keep = dropout_keep(T, h, p, seed, token_offset)
    out = _rb(X + np.where(keep, (O @ Wo + bo) * dropout_scale(p), 0.0), mirror)
    return {"QKV": QKV, "QKr": np.concatenate([x.reshape(T, h) for x in turned], axis=1), "P": P, "O": O, "out": out, "keep": keep}


def bwd(dOut, X, Wqkv, Wo, fw, nh, seq_len, p, rope, mirror=False):
    T, h = X.shape
    d = h // nh
    QKV, P, O, keep = fw["QKV"], fw["P"], fw["O"], fw["keep"]
    q, k, v = _heads(fw["QKr"][:, :h], nh), _heads(fw["QKr"][:, h:], nh), _heads(QKV[:, 2 * h:], nh)
    dZ = _rb(np.where(keep, dOut * dropout_scale(p), 0.0), mirror)
    dO = _heads(_rb(dZ @ Wo.T, mirror), nh)
    g = np.empty((3, T, nh, d))
    for s in range(T // seq_len):
        r = slice(s * seq_len, (s + 1) * seq_len)
        for j in range(nh):
            pr, do = P[s, j], dO[r, j]
            dp = do @ v[r, j].T
            ds = _rb(pr * (dp - (dp * pr).sum(axis=1, keepdims=True)) / math.sqrt(d), mirror)
            g[0, r, j], g[1, r, j], g[2, r, j] = ds @ k[r, j], ds.T @ q[r, j], pr.T @ do
    g = _rb(g, mirror)
    dws = []
    for i, w in ((0, rope["wq"]), (1, rope["wk"])):
        g[i], dw = qro.bwd(_heads(QKV[:, i * h:(i + 1) * h], nh), w, g[i].copy(), rope["ang"], rope["rot"], rope["inter"], rope["eps"])
        dws.append(dw)
    dQKV = _rb(np.concatenate([x.reshape(T, h) for x in g], axis=1), mirror)
    return {"dQKV": dQKV, "dX": _rb(dOut + dQKV @ Wqkv.T, mirror), "dWqkv": X.T @ dQKV, "dbqkv": dQKV.sum(axis=0),
            "dWo": O.T @ dZ, "dbo": dZ.sum(axis=0), "dwq": dws[0], "dwk": dws[1]}
