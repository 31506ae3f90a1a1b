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
