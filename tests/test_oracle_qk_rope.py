"""Pins of the oracle of the head norms with rotation."""
import numpy as np
import pytest
import torch

from oracle import qk_rope_oracle as qro

FORMS = [(16, 16, False, [8]), (16, 16, True, [4, 4]), (24, 8, False, [2, 1, 1]), (24, 16, True, [3, 0, 5])]


def _case(d, rot, sections, T=5, n=3, seed=1):
    rng = np.random.default_rng(seed)
    pos = rng.integers(-50, 2000, (len(sections), T))
    inv = rng.uniform(1e-3, 1.0, rot // 2).astype(np.float32)
    return rng.standard_normal((T, n, d)), 1 + 0.3 * rng.standard_normal(d), qro.angles(pos, inv, sections), rng.standard_normal((T, n, d))


@pytest.mark.parametrize("d,rot,inter,sections", FORMS)
def test_rotation_keeps_norms_and_sees_differences_only(d, rot, inter, sections):
    x, _, ang, y = _case(d, rot, sections)
    tx = qro.turn(x, ang, rot, inter)
    np.testing.assert_allclose((tx**2).sum(-1), (x**2).sum(-1), rtol=1e-12)
    np.testing.assert_array_equal(tx[..., rot:], x[..., rot:])
    # <turn(x, s), turn(y, t)> = <x, turn(y, t - s)>
    other = ang[::-1].copy()
    np.testing.assert_allclose((tx * qro.turn(y, other, rot, inter)).sum(-1),
                               (x * qro.turn(y, other - ang, rot, inter)).sum(-1), rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("d,rot,inter,sections", FORMS)
def test_against_autograd(d, rot, inter, sections, norm):
    x, w, ang, dy = _case(d, rot, sections)
    xt = torch.tensor(x, requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    n = xt * torch.rsqrt((xt * xt).mean(-1, keepdim=True) + 1e-5) * wt if norm else xt
    c, s = (torch.tensor(f(ang))[:, None] for f in (np.cos, np.sin))
    r = n[..., :rot]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    y = torch.cat([r, n[..., rot:]], -1)
    y.backward(torch.tensor(dy))
    np.testing.assert_allclose(qro.fwd(x, w if norm else None, ang, rot, inter, 1e-5), y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw = qro.bwd(x, w if norm else None, dy, ang, rot, inter, 1e-5)
    np.testing.assert_allclose(dx, xt.grad.numpy(), rtol=1e-10, atol=1e-10)
    if norm:
        np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-10, atol=1e-10)
    else:
        assert dw is None


def test_central_differences():
    d, rot, inter, sections = FORMS[2]
    x, w, ang, dy = _case(d, rot, sections)
    dx, dw = qro.bwd(x, w, dy, ang, rot, inter, 1e-5)
    v, u = np.random.default_rng(4).standard_normal(x.shape), np.random.default_rng(5).standard_normal(d)
    f = lambda e: (qro.fwd(x + e * v, w + e * u, ang, rot, inter, 1e-5) * dy).sum()  # noqa: E731
    want = (dx * v).sum() + (dw * u).sum()
    assert abs((f(1e-6) - f(-1e-6)) / 2e-6 - want) <= 1e-6 * (1 + abs(want))
