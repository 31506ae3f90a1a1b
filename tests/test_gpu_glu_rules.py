"""The gated block at both sides of the limit beyond which its second product leaves the few-token
launch: the outputs of a quarter of the 152 SMs' tiles, 38 * 256 * 256 = 1216 * 2048."""
import pytest
import torch

import test_gpu_glu as glu
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


@pytest.mark.parametrize("T", [1216, 1217])
def test_outputs_at_the_limit_of_the_few_token_launch(T):
    h, ffn = 2048, 72
    c = glu.Case(T, h, ffn)
    (GU, gu), (Y, y), (O, o) = glu._guarded(T, 2 * ffn), glu._guarded(T, ffn), glu._guarded(T, h)
    c.fwd(GU, Y, O)
    glu._status_ok()
    glu.check_forward(c, GU, Y, O)
    (dZ, z), (dGU, dgu), (dX, dx) = glu._guarded(T, h), glu._guarded(T, 2 * ffn), glu._guarded(T, h)
    c.bwd_input(GU, dZ, dGU, dX)
    glu._status_ok()
    glu.check_backward_input(c, GU, dZ, dGU, dX)
    for behind in (gu, y, o, z, dgu, dx):
        assert torch.all(behind == 7)
