"""Head norms with rotation where a lane of a warp has no head, and where values are not finite.

Bounds are those of test_gpu_qk_rope, which hold for any eps; eps = 0 is taken with random heads, none
of which is all zeros.
"""
import pytest
import torch

import test_gpu_qk_rope as qk
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,nq,nk,d,rot", [
    (5, 1, 2, 128, 128),        # four heads to a warp
    (3, 128, 128, 160, 160),    # three
    (7, 5, 3, 72, 40),          # three, vectors of four elements
    (700, 3, 1, 256, 64),       # two
    (2, 31, 33, 8, 8),          # 32
])
def test_eps_zero_and_heads_that_leave_part_of_a_warp(T, nq, nk, d, rot, inter, monkeypatch):
    """The weights' gradients sum over the heads that there are, and over nothing else."""
    monkeypatch.setattr(qk, "EPS", 0.0)
    c = qk.Case(T, nq, nk, d, rot, inter)
    c.kw["eps"] = 0.0
    (Qo, _), (Ko, _), (dQ, _), (dK, _) = c.out(nq), c.out(nk), c.out(nq), c.out(nk)
    c.fwd(Qo, Ko)
    qk._status_ok()
    qk.check_fwd(c, Qo, Ko)
    w = c.grads()
    c.bwd(dQ, dK, w)
    qk._status_ok()
    qk.check_bwd(c, dQ, dK, w)


def _same(a, b):
    return bool(torch.all((a == b) | (torch.isnan(a) & torch.isnan(b))))


BEHIND = [(3, 5, 2, 128, 64, False), (3, 5, 2, 128, 64, True), (4, 3, 1, 72, 40, False), (4, 3, 1, 72, 40, True), (2, 2, 2, 256, 16, False)]


@pytest.mark.parametrize("T,nq,nk,d,rot,inter", BEHIND)
def test_elements_behind_rot_keep_to_themselves(T, nq, nk, d, rot, inter):
    """The rotation alone, forwards and back, moves no element behind `rot` and lets none of them, infinite
    or NaN, into another."""
    c = qk.Case(T, nq, nk, d, rot, inter, norm=False)
    for t in (c.Q, c.K, c.dQo, c.dKo):
        for i, v in enumerate((float("inf"), float("-inf"), float("nan"))):
            t[i % T, i % t.shape[1], rot + 5 * i] = v
        t[T - 1, 0, d - 1] = float("inf")
    ins = (c.Q, c.K, c.dQo, c.dKo)
    outs = [c.out(n)[0] for n in (nq, nk, nq, nk)]
    c.fwd(*outs[:2])
    c.bwd(*outs[2:], c.grads())
    zeroed = [t.clone() for t in ins]
    for t in zeroed:
        t[..., rot:] = 0
    clean = [c.out(n)[0] for n in (nq, nk, nq, nk)]
    c.fwd(*clean[:2], Q=zeroed[0], K=zeroed[1])
    c.bwd(*clean[2:], c.grads(), dQo=zeroed[2], dKo=zeroed[3])
    qk._status_ok()
    for x, y, z in zip(ins, outs, clean):
        assert _same(y[..., rot:], x[..., rot:])
        assert torch.equal(y[..., :rot], z[..., :rot])


@pytest.mark.parametrize("T,nq,nk,d,rot,inter", BEHIND)
def test_an_infinity_behind_rot_with_the_norm(T, nq, nk, d, rot, inter):
    """Forwards, an infinite element's head has an infinite norm: its other elements are zeros, and the
    element itself, inf / inf, is NaN.  Backwards, an infinite gradient there reaches every dx of its head
    by the mean, but of dw only its own element."""
    c = qk.Case(T, nq, nk, d, rot, inter)
    at = rot + 3
    x = c.Q.clone()
    x[1, 1, at] = float("inf")
    (Qo, _), (Ko, _), (dQ, _), (dK, _) = c.out(nq), c.out(nk), c.out(nq), c.out(nk)
    c.fwd(Qo, Ko, Q=x)
    g = c.dQo.clone()
    g[1, 1, at] = float("-inf")
    w = c.grads()
    c.bwd(dQ, dK, w, dQo=g)
    qk._status_ok()
    bad = torch.isnan(Qo)
    assert bad.sum() == 1 and bool(bad[1, 1, at])
    assert torch.all(Qo[1, 1][~bad[1, 1]] == 0)
    ok = torch.isfinite(w["dwq"])
    assert (~ok).sum() == 1 and not bool(ok[at]) and torch.isfinite(w["dwk"]).all()
    ok = torch.isfinite(dQ).all(-1)
    assert (~ok).sum() == 1 and not bool(ok[1, 1]) and torch.isfinite(dK).all()
