"""GPU parity of the 8-bit key/value cache in every kernel that its launch rules choose from.

The rules are restated here, so that a case that no longer reaches its kernel fails.  Bounds are those of test_gpu_kv_cache.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_gpu_kv_cache import Attn, Pool, _rows, _slots, _status_ok, check_write, i32

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


def write_launch(tokens, nk, bs):
    """(chunk, span) of kv_write: the tokens that a CTA looks through for runs, and the heads of keys and values that it takes."""
    heads, full = 2 * nk, torch.cuda.get_device_properties(0).multi_processor_count * (512 // bs)
    chunk = 1
    while chunk < bs and tokens * heads >= full * chunk:
        chunk *= 2
    return chunk, max(1, min(-(-tokens // chunk) * heads // full, 8))


# Key heads, so that a span begins with keys and ends with values, and the last one is not full.
@pytest.mark.parametrize("bs,nk,d,tokens,span", [
    (16, 45, 32, 3800, 4), (16, 131, 32, 2600, 8), (32, 65, 64, 2050, 3), (32, 49, 224, 2800, 3), (64, 33, 160, 2700, 2), (64, 131, 32, 2600, 8),
    (16, 35, 128, 5000, 4), (64, 67, 96, 2000, 3)])
def test_write_several_heads_a_cta(bs, nk, d, tokens, span):
    """Whole blocks, parts of them, runs of a few tokens and single ones in any order, rows without a slot between them, over codes
    that move."""
    rng = np.random.default_rng(bs + nk)
    runs, count = [], 0
    while count < tokens:
        off = int(rng.integers(0, bs))
        n = int(rng.choice([1, 2, 7, bs, bs]))
        if n == bs:
            off = int(rng.choice([0, off]))
        n = min(n, bs - off, tokens - count)
        runs.append((len(runs), off, n))
        count += n
        if rng.random() < 0.1 and count < tokens:
            runs.append(None)
            count += 1
    order = rng.permutation(len(runs))
    runs = [r if r is None else (int(order[r[0]]), r[1], r[2]) for r in runs]
    slots = _slots(runs, bs)
    assert len(slots) == tokens and write_launch(tokens, nk, bs) == (bs, span)
    assert nk % span != 0 and (2 * nk % span != 0 or span == 2)
    pool = Pool(len(runs), nk, bs, d)
    K, V = _rows(tokens, nk, d, 16, 1, 2.0), _rows(tokens, nk, d, 0, 2)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


@pytest.mark.parametrize("bs,nk,tokens,chunk", [(16, 3, 5, 1), (64, 8, 600, 8), (32, 40, 2500, 32), (64, 3, 20000, 64)])
def test_write_every_chunk(bs, nk, tokens, chunk):
    """Prompts over whole blocks, one after another, for every number of tokens that a CTA looks through."""
    assert write_launch(tokens, nk, bs)[0] == chunk
    blocks = -(-tokens // bs) + 1
    order = np.random.default_rng(nk).permutation(blocks)
    slots = np.concatenate([b * bs + np.arange(bs) for b in order])[:tokens].astype(np.int32)
    pool = Pool(blocks, nk, bs, 64)
    K, V = _rows(tokens, nk, 64, 0, 1), _rows(tokens, nk, 64, 8, 2)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


@pytest.mark.parametrize("d,large", [(64, 3), (160, 2)])
def test_attn_of_the_rows_that_there_are_and_of_a_whole_buffer(d, large):
    """A buffer of 72 rows for 4 single tokens makes for larger tiles, its first 4 rows for those of one token."""
    c = Attn([2000, 5, 0, 333], [1, 1, 1, 1], 16, 4, d, 32, pad=68)
    assert tile(72, 4, 4, d) == large and tile(4, 4, 4, d) == 1
    c.run()
    _status_ok()
    c.check()
    c.O.fill_(7.0)
    mlp.kv_attn(c.Q[:4], *c.pool.dev, c.dt, c.dl, c.dc, c.O[:4], c.ws)
    _status_ok()
    c.check()


@pytest.mark.parametrize("n", [127, 128, 129, 255, 256, 257, 384])
@pytest.mark.parametrize("long", [128, 1000])
def test_attn_requests_about_whole_groups(n, long):
    """The work is counted in groups of 128 requests: equal ones, whose shares may end where a group does, the last of a group long."""
    lens = [128] * n
    lens[min(127, n - 1)] = lens[-1] = long
    c = Attn(lens, [1] * n, 2, 1, 32, 16, seed=n)
    c.run()
    _status_ok()
    c.check()


FRESH = """
import sys, threading
sys.path[:0] = [".", "tests"]
import torch
import test_gpu_kv_cache as kv
from transformer_lm_megatron_gb300 import mlp

mlp.load()
# heads and rows for a kernel of each kind: tiles of 8, 16 and 24 rows, and the write's block sizes
CASES = [(64, 1, 1, 16), (96, 9, 1, 32), (128, 24, 1, 64), (160, 5, 1, 16), (256, 2, 6, 64)]


def work(seed, stream, start):
    with torch.cuda.stream(stream):
        made = [(kv.Attn([700, 33], [new] * 2, 2 * group, 2, d, bs, seed=seed + d), kv._rows(19, 2, d, 0, seed)) for d, group, new, bs in CASES]
        got = []
        for c, K in made:
            start()
            mlp.kv_write(K, K, torch.arange(19, dtype=torch.int32, device="cuda"), *c.pool.dev)
            start()
            c.run()
            got += [c.O, *c.pool.dev]
        stream.synchronize()
        return [t.clone() for t in got]


streams = [torch.cuda.Stream() for _ in range(2)]
barrier, outs = threading.Barrier(2, timeout=120), {}
threads = [threading.Thread(target=lambda k=k: outs.__setitem__(k, work(k + 1, streams[k], barrier.wait))) for k in range(2)]
[t.start() for t in threads]
[t.join() for t in threads]
for k in range(2):
    alone = work(k + 1, streams[k], lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(alone, outs[k])), k
assert mlp.mlp_sync_status() == 0
print("FIRST CALLS OK")
"""


def test_first_calls_from_two_threads():
    """What a first launch works out is worked out once, whichever thread comes first."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "FIRST CALLS OK" in r.stdout, r.stdout + r.stderr
