"""GPU parity of the attention over the 8-bit cache where value maxima lie far apart.

Bounds are those of test_gpu_kv_cache.
"""
import numpy as np
import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_gpu_kv_cache import Attn, _status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


def _values(c, most, zero):
    """Value maxima `most` [blocks, nk], and blocks of zeros where `zero`."""
    c.pool.Vmax[:] = np.where(zero, 0, most)
    c.pool.Vc[zero] = 0
    c.pool.dev[1].copy_(torch.from_numpy(c.pool.Vc))
    c.pool.dev[3].copy_(torch.from_numpy(c.pool.Vmax))


@pytest.mark.parametrize("qscale", [0.01, 0.3, 3.0])
@pytest.mark.parametrize("most", [2.0**10, 2.0**36, 2.0**50, 2.0**70, 2.0**115, 255 * 2.0**120, 2.0**-60])
@pytest.mark.parametrize("first", [False, True])
def test_attn_many_blocks_of_zeros_beside_large_values(most, qscale, first):
    """Blocks of zeros hold half of the tokens, before or between the others: their weights count in the softmax's sum, however
    large the other values are."""
    c = Attn([900, 4000], [1, 2], 8, 2, 64, 16, qscale=qscale)
    zero = np.zeros(c.pool.Vmax.shape, bool)
    for r in range(2):
        k = -(-int(c.lens[r]) // 16)
        zero[c.table[r, : k // 2] if first else c.table[r, 0:k:2]] = True
    _values(c, most, zero)
    c.run()
    _status_ok()
    c.check()


@pytest.mark.parametrize("d,group,new", [(32, 2, 1), (64, 4, 5), (128, 8, 1), (128, 5, 5), (160, 1, 1), (256, 4, 3)])
@pytest.mark.parametrize("far", [1, 7, 40])
def test_attn_value_maxima_over_all_of_the_range(d, group, new, far):
    """Maxima from 2^-79 to 2^120, each block's by chance, or most of them small and every `far`-th one large; requests over
    several CTAs, whose parts have bases 2^200 apart."""
    c = Attn([3000, 40, 700], [new] * 3, 2 * group, 2, d, 16, seed=d + far)
    rng = np.random.default_rng(far)
    most = np.exp2(rng.integers(-79, 121, c.pool.Vmax.shape) if far == 1 else rng.integers(-79, 0, c.pool.Vmax.shape))
    if far > 1:
        most[c.table[0, ::far]] = 2.0**100
    _values(c, most, np.zeros(c.pool.Vmax.shape, bool))
    c.run()
    _status_ok()
    c.check()
