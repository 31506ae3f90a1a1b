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


def test_write_codes_of_every_pair_of_significands():
    """Every value x against every maximum, x's exponent up to 9 below: the codes are rint(127 x / max), ties included."""
    m = np.arange(128, 256, dtype=np.float64)
    x = (m[None, :] * 2.0 ** -np.arange(10.0)[:, None]).reshape(-1)  # 1280 values
    rows = np.zeros((128, 16, 96))
    for i, top in enumerate(m):
        rows[i].reshape(-1)[: len(x)] = np.where(x <= top, x, 0)
        rows[i, 15, 95] = top
    K = torch.from_numpy(rows.reshape(128 * 16, 1, 96)).to(torch.bfloat16).cuda()
    V = -K * 2.0**-79 * 2.0**-7  # maxima from 2^-79 on, negative
    pool, slots = Pool(128, 1, 16, 96), np.arange(128 * 16, dtype=np.int32)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)
    np.testing.assert_array_equal(pool.dev[0].cpu().numpy(), np.rint(rows * 127 / m[:, None, None])[:, None].astype(np.int8))


@pytest.mark.parametrize("at", [2.0**-7, 2.0**120, 2.0**-77])
def test_write_moves_every_code_between_every_pair_of_significands(at):
    """All codes of a block from every maximum to every larger one, its exponent up to 8 above: rint(code * old / new)."""
    m = np.arange(128, 256, dtype=np.float64)
    gaps = 2.0 ** -np.arange(9.0)
    old = (m[:, None] * gaps).reshape(-1, 1) * np.ones(128) * at  # [1152 blocks, 128 heads]
    new = np.broadcast_to(m * at, old.shape)
    codes = np.zeros((16, 32), np.int8)
    codes[:8].reshape(-1)[:255] = np.arange(-127, 128)
    held = torch.from_numpy(codes).cuda().expand(1152, 128, 16, 32)
    Kc, Vc = held.clone(), held.clone()
    Kmax, Vmax = (torch.from_numpy(old.astype(np.float32)).cuda() for _ in range(2))
    K = torch.zeros(1152, 128, 32, dtype=torch.float64)
    K[:, :, 3] = torch.from_numpy(np.ascontiguousarray(new))
    K = K.to(torch.bfloat16).cuda()
    V = torch.zeros_like(K)
    mlp.kv_write(K, V, i32(np.arange(1152) * 16 + 8), Kc, Vc, Kmax, Vmax)
    _status_ok()
    top = torch.from_numpy(np.maximum(old, new)).cuda()
    assert torch.equal(Kmax.double(), top)
    want = held.double() * torch.from_numpy(old).cuda()[..., None, None]  # exact: 8 bits times 7
    want = torch.round(want / top[..., None, None])  # (fp64's rounding is 2^-45 of a code, no quotient is so near a tie)
    want[:, :, 8] = 0
    want[:, :, 8, 3] = torch.round(127 * torch.from_numpy(np.ascontiguousarray(new)).cuda() / top)
    assert torch.equal(Kc, want.to(torch.int8))
    held = held.clone()
    held[:, :, 8] = 0
    assert torch.equal(Vc, held) and torch.equal(Vmax.double(), torch.from_numpy(old).cuda())
