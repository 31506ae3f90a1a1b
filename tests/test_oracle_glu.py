"""Pins of the gated block's oracle: autograd in float64, slices, central differences."""
import numpy as np
import pytest
import torch

from oracle import glu_oracle as glo


def _case(T=6, h=16, ffn=24, seed=3):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(X=r(T, h), A=0.4 * r(h, 2 * ffn), a=r(2 * ffn), B=0.4 * r(ffn, h), b=r(h), dO=r(T, h))


def _forward(c, kind, p=0.2, t=1):
    GU = glo.gates(c["X"], c["A"], c["a"], t)
    Y = glo.gated(GU, kind)
    return GU, Y, glo.out(Y, c["B"], c["b"], c["X"], p, 1234, 5, t)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_against_autograd(kind):
    c = _case()
    leaf = {k: torch.tensor(c[k], requires_grad=True) for k in ("X", "A", "a", "B", "b")}
    GU = leaf["X"] @ leaf["A"] + leaf["a"]
    f = GU.shape[1] // 2
    gate = torch.nn.functional.silu(GU[:, :f]) if kind == "silu" else torch.nn.functional.gelu(GU[:, :f], approximate="tanh")
    Z = (gate * GU[:, f:]) @ leaf["B"] + leaf["b"]
    keep = torch.tensor(glo.dropout_keep(6, 16, 0.2, 1234, 5))
    O = leaf["X"] + torch.where(keep, Z * glo.dropout_scale(0.2), 0.0)
    O.backward(torch.tensor(c["dO"]))
    GUo, Y, Oo = _forward(c, kind)
    np.testing.assert_allclose(Oo, O.detach().numpy(), rtol=1e-12, atol=1e-12)
    dZ = glo.d_out(c["dO"], 0.2, 1234, 5)
    dGU = glo.d_gates(dZ, c["B"], GUo, kind)
    dA, da, dB, db = glo.d_weights(c["X"], dZ, Y, dGU)
    for name, got in (("X", glo.d_input(dGU, c["A"], c["dO"])), ("A", dA), ("a", da), ("B", dB), ("b", db)):
        np.testing.assert_allclose(got, leaf[name].grad.numpy(), rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_slices_change_nothing(kind):
    c = _case()
    for t in (2, 3):
        for x, y in zip(_forward(c, kind, t=1), _forward(c, kind, t=t)):
            np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_central_differences(kind):
    c = _case(T=3, h=8, ffn=8)
    GU, Y, _ = _forward(c, kind)
    dZ = glo.d_out(c["dO"], 0.2, 1234, 5)
    dGU = glo.d_gates(dZ, c["B"], GU, kind)
    dA, da, dB, db = glo.d_weights(c["X"], dZ, Y, dGU)
    grads = dict(X=glo.d_input(dGU, c["A"], c["dO"]), A=dA, a=da, B=dB, b=db)
    rng = np.random.default_rng(0)
    for name, g in grads.items():
        v = rng.standard_normal(g.shape)
        e = 1e-6
        loss = lambda s: (_forward({**c, name: c[name] + s * v}, kind)[2] * c["dO"]).sum()  # noqa: E731, B023
        assert abs((loss(e) - loss(-e)) / (2 * e) - (g * v).sum()) <= 1e-6 * (1 + abs((g * v).sum())), name
