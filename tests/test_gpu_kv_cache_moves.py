"""GPU parity of the cache write where the codes of a block move to a larger maximum: maxima near the end of fp32's range, and
every pair of significands."""
import numpy as np
import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_gpu_kv_cache import Pool, _slots, _status_ok, check_write, i32

pytestmark = pytest.mark.gpu

LARGEST = 255 * 2.0**120  # of bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


# (a short run is one of 64 pieces of 16 bytes or fewer: a token of any head size; ten tokens of 128 are a long one)
@pytest.mark.parametrize("d,count", [(32, 1), (128, 10), (256, 1)])
@pytest.mark.parametrize("old,new", [(2.0**119, 1.5 * 2.0**119), (2.0**120, 129 * 2.0**113), (2.0**121, 2.0**122), (2.0**124, 2.0**126),
                                     (254 * 2.0**120, LARGEST), (2.0**122, LARGEST), (2.0**-70, LARGEST), (2.0**-126, LARGEST)])
def test_write_moves_codes_to_a_huge_maximum(old, new, d, count):
    """code * old leaves fp32 above 2^121, where bf16 does not: the codes before move all the same."""
    pool = Pool(4, 2, 16, d)
    pool.Kmax[:], pool.Vmax[:] = old, old
    pool.dev = [torch.from_numpy(x).cuda() for x in (pool.Kc, pool.Vc, pool.Kmax, pool.Vmax)]
    slots = _slots([(2, 5, count), (0, 3, 1)], 16)
    g = torch.Generator().manual_seed(d)
    K, V = ((torch.rand(len(slots), 2, d, generator=g, dtype=torch.float64) * 2 - 1) * new for _ in range(2))
    K[:, :, 1], V[:, :, d - 1] = new, -new
    K, V = K.to(torch.bfloat16).cuda(), V.to(torch.bfloat16).cuda()
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)
