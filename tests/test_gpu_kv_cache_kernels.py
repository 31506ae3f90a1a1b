"""GPU parity of the 8-bit key/value cache in every kernel that its launch rules choose from.

The rules are restated here, so that a case that no longer reaches its kernel fails.  Bounds are those of test_gpu_kv_cache.
"""
import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_gpu_kv_cache import Attn, _rows, _status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


def tile(rows, n, group, d):
    """Eights of rows of kv_attn's tiles, for a request's rows on average."""
    each = -(-rows // n) * group
    if each <= 8:
        return 1
    return 3 if d <= 128 and -(-each // 24) * 5 < -(-each // 16) * 4 else 2


TILES = [  # query heads to a key head, new tokens of each request, eights of a tile's rows for heads up to 128 and above
    (1, 1, 1, 1), (8, 1, 1, 1), (2, 3, 1, 1), (5, 1, 1, 1), (1, 8, 1, 1), (9, 1, 2, 2), (16, 1, 2, 2), (4, 4, 2, 2), (5, 5, 2, 2), (6, 4, 3, 2), (8, 5, 3, 2),
    (12, 6, 3, 2)]


@pytest.mark.parametrize("group,new,small,large", TILES)
@pytest.mark.parametrize("d", range(32, 257, 32))
def test_attn_every_head_size_and_tile(d, group, new, small, large):
    """Requests that are cut among CTAs (93 steps of 16 tokens and more), short ones, and one of whole steps; Q's and O's rows apart
    by strides of their own."""
    lens = [1500, new, 90, 2048, 16]
    c = Attn(lens, [new] * 5, 2 * group, 2, d, 16, gap=8, seed=d + 10 * group + new)
    nt = tile(c.T, 5, group, d)
    assert nt == (small if d <= 128 else large)
    # A tile counts its steps and 16 more, a CTA (there are two an SM at least) gets an equal share: one shorter than what is
    # between the first 8 and the last 8 steps of the long requests' tiles cuts each of them.
    work = 2 * -(-new * group // (8 * nt)) * sum(-(-n // 16) + 16 for n in lens)
    assert -(-work // (2 * torch.cuda.get_device_properties(0).multi_processor_count)) < 1500 // 16 - 2 * 8
    c.Q = _rows(c.T, 2 * group, d, 24, d)
    c.run()
    _status_ok()
    c.check()


@pytest.mark.parametrize("d", [128, 160, 256])
def test_attn_a_block_size_of_every_kind_in_the_tile_of_eight_rows(d):
    for bs in (16, 32, 64):
        c = Attn([3000, 17, 333], [1, 1, 1], 8, 1, d, bs, seed=bs)
        assert tile(c.T, 3, 8, d) == 1
        c.run()
        _status_ok()
        c.check()
