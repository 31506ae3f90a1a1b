"""The 8-bit key/value cache as a serving loop uses it over many steps: drafts of which some are refused, requests that end and
others that take their place, blocks that go back to the free list; and beside the attention block that it answers for.

Bounds are those of test_gpu_kv_cache where no others are given.
"""
import numpy as np
import pytest
import torch

from oracle import kv_cache_oracle as kvo
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from gpu_harness import BF16_TOL, to_f64
from test_gpu_decoder_layer import Layer
from test_gpu_kv_cache import Loop, _status_ok, i32, largest, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


def give_back(table, lens, new_lens, free, taken, bs):
    """The free list and its count after requests went from lens to new_lens tokens (include/gb_mlp.h, kv_plan)."""
    free = free.copy()
    for r in range(len(lens)):
        for b in range(-(-int(new_lens[r]) // bs), -(-int(lens[r]) // bs)):
            taken -= 1
            free[taken] = table[r, b]
    return free, taken


@pytest.mark.parametrize("bs", [16, 32])
def test_drafts_that_are_refused_and_requests_that_end(bs):
    """A pool with hardly more blocks than are held at once: lost ones would leave the loop without any."""
    n, nq, nk, d, rows, blocks = 5, 8, 2, 64, 5 * 45, 5 * 6
    L = Loop(n, nq, nk, d, bs, width=6, blocks=blocks, rows=rows)
    rng, g = np.random.default_rng(bs), torch.Generator().manual_seed(bs)
    lens, table, taken, free = np.zeros(n, np.int32), L.table.cpu().numpy(), 0, L.free.cpu().numpy()
    codes = [np.zeros((blocks, nk, bs, d), np.int8) for _ in range(2)]
    most = [np.zeros((blocks, nk)) for _ in range(2)]
    given, begun = 0, 0
    for k in range(24):
        # requests that end or take drafts back, by the host
        kept = lens.copy()
        if k > 0:
            back = rng.integers(0, 5, n)  # of at most five drafts at least one is kept
            kept = np.where((lens > 70) | (rng.random(n) < 0.08), 0, np.where(drafted, lens - np.minimum(back, add - 1), lens)).astype(np.int32)
            free, now = give_back(table, lens, kept, free, taken, bs)
            given, taken, lens = given + taken - now, now, kept
            L.lens[k % 2].copy_(torch.from_numpy(lens))
            L.free.copy_(torch.from_numpy(free))
            L.taken[k % 2].fill_(taken)
        # a slot without a request gets a prompt, the others a token or five drafts
        begun += int((lens == 0).sum())
        drafted = lens > 0
        add = np.where(lens == 0, rng.integers(1, 41, n), rng.choice([1, 5], n)).astype(np.int32)
        L.add.copy_(torch.from_numpy(add))
        L.QKV.copy_((torch.randn(L.QKV.shape, generator=g) * float(rng.uniform(0.5, 2))).to(torch.bfloat16))
        L.O.fill_(7.0)
        L.step(k)
        _status_ok()
        status, lens, taken, cu, pos, slots, table = kvo.plan(add, lens, table, free, taken, bs, rows)
        assert status == 0 and int(L.status) == 0 and int(L.taken[1 - k % 2]) == taken
        np.testing.assert_array_equal(L.slots.cpu().numpy(), slots)
        np.testing.assert_array_equal(L.table.cpu().numpy(), table)
        held = [int(b) for r in range(n) for b in table[r, : -(-int(lens[r]) // bs)]]
        assert len(set(held)) == len(held) == taken and not set(held) & set(free[taken:].tolist())  # no block lost, none twice
        Kr, V = to_f64(L.Kr.cpu()), to_f64(L.V.cpu())
        for i, (x, c, m) in enumerate(((Kr, L.cache.Kc, L.cache.Kmax), (V, L.cache.Vc, L.cache.Vmax))):
            codes[i], most[i] = kvo.write(x, slots, codes[i], most[i])
            np.testing.assert_array_equal(c.cpu().numpy(), codes[i])
            np.testing.assert_array_equal(m.cpu().numpy().astype(np.float64), most[i])
        q, got = to_f64(L.Qr.cpu()), to_f64(L.O.cpu())
        for r in range(n):
            at = slice(int(cu[r]), int(cu[r + 1]))
            o, A, E = kvo.attn(q[at], codes[0], codes[1], most[0], most[1], table[r], int(lens[r]), float(np.float32(d**-0.5)))
            assert bool((np.abs(got[at] - o) <= tolerance(o, A, E, int(lens[r]), largest(most[1], table[r], int(lens[r]), bs))).all())
        assert bool((got[int(cu[n]) :] == 7).all())
    assert given >= 15 and begun > 8  # (so many came to pass)


def test_a_refused_token_that_is_not_finite():
    """It leaves the block that it was in reading as NaN until that is begun anew; a block that it began goes back and forgets it."""
    bs, d = 16, 64
    cache = mlp.KVCache(3, 1, bs, d)
    pool = (cache.Kc, cache.Vc, cache.Kmax, cache.Vmax)
    g = torch.Generator().manual_seed(1)
    x = lambda t: torch.randn(t, 1, d, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    mlp.kv_write(x(15), x(15), i32(range(15)), *pool)
    bad = x(2)
    bad[:, 0, 3] = float("nan")
    mlp.kv_write(bad, bad, i32([15, 16]), *pool)  # the last place of block 0, the first of block 1
    _status_ok()
    assert torch.isnan(cache.Kmax[:2]).all() and torch.isnan(cache.Vmax[:2]).all()
    K = x(2)
    mlp.kv_write(K, K, i32([15, 16]), *pool)  # both refused, others come
    _status_ok()
    assert torch.isnan(cache.Kmax[0]).all() and torch.equal(cache.Kmax[1, 0], K[1].abs().max().float())
    mlp.kv_write(x(1), x(1), i32([0]), *pool)
    _status_ok()
    assert bool(torch.isfinite(cache.Kmax[0]).all())


@pytest.mark.parametrize("bs", [16, 64])
def test_keys_and_values_of_the_attention_block(bs):
    """attn_rope_fwd's rotated keys and its values go into the cache as prompts, single tokens and drafts; each step's attention is
    the block's own over the tokens so far.

    A value is off by at most (1 + its block's growths) max / 254 (include/gb_mlp.h): dv, and keys by dk.  A score is off by
    e = sum |q| dk / sqrt(d) then, a softmax weight by a factor within exp(+-2 e): |got - o| <= A (exp(2 e) - 1) + dv and the kernel's
    own bound; the block's O is held to BF16_TOL of its largest.
    """
    h, nh, L = 256, 4, 128
    d, n, T = h // nh, 2, 2 * L
    layer = Layer(T, h, nh, L, 32, False, (16,), True)
    g = torch.Generator().manual_seed(bs)
    layer.fwd(torch.randn(T, h, generator=g).to(torch.bfloat16).cuda())
    heads = lambda x: x.view(n, L, nh, d)  # noqa: E731
    Q, K, V = layer.QKr[:, :h].view(T, nh, d), layer.QKr[:, h:].view(T, nh, d), layer.buf.QKV[:, 2 * h :].view(T, nh, d)
    block = to_f64(layer.buf.O.cpu()).reshape(n, L, nh, d)
    q64, k64, v64 = (heads(torch.from_numpy(to_f64(x.cpu().contiguous()))).numpy() for x in (Q, K, V))
    blocks = n * (L // bs)
    cache = mlp.KVCache(blocks, nh, bs, d)
    table, free = torch.full((n, L // bs), -1, dtype=torch.int32, device="cuda"), i32(np.random.default_rng(bs).permutation(blocks))
    lens, taken = [i32([0, 0]), i32([0, 0])], [i32([0]), i32([0])]
    ws, have, k = torch.empty(mlp.kv_attn_workspace(d), device="cuda"), np.zeros(n, int), 0
    grown = [np.zeros((blocks, nh)) for _ in range(2)]  # how often a block's maximum grew after it had tokens, Kmax and Vmax
    rng = np.random.default_rng(1)
    while have.min() < L:
        add = np.array([41, 75]) if k == 0 else np.minimum(rng.choice([0, 1, 1, 5], n), L - have)
        if add.sum() == 0:
            continue
        at = np.concatenate([r * L + np.arange(have[r], have[r] + add[r]) for r in range(n)])
        rows = len(at)
        cu, pos, slots, status = i32(np.zeros(n + 1)), i32(np.zeros(rows)), i32(np.zeros(rows)), i32([1])
        mlp.kv_plan(i32(add), lens[k % 2], table, free, taken[k % 2], bs, lens[1 - k % 2], taken[1 - k % 2], cu, pos, slots, status)
        before = [x.clone() for x in (cache.Kmax, cache.Vmax)]
        mlp.kv_write(K[at], V[at], slots, cache.Kc, cache.Vc, cache.Kmax, cache.Vmax)
        O = torch.empty(rows, nh, d, dtype=torch.bfloat16, device="cuda")
        mlp.kv_attn(Q[at], cache.Kc, cache.Vc, cache.Kmax, cache.Vmax, table, lens[1 - k % 2], cu, O, ws)
        _status_ok()
        assert int(status) == 0
        for i, (old, new) in enumerate(zip(before, (cache.Kmax, cache.Vmax))):
            grown[i] += ((old > 0) & (new > old)).cpu().numpy()
        have, k = have + add, k + 1
        got, at_row = to_f64(O.cpu()), 0
        for r in range(n):
            tab = table[r].cpu().numpy()
            off = []  # of each token and head: the most that its key and its value may be off
            for i, most in enumerate((cache.Kmax, cache.Vmax)):
                step = (1 + grown[i]) * most.cpu().numpy().astype(np.float64) / 254
                off.append(step[tab[np.arange(have[r]) // bs]])
            held = []
            for codes, most, x in ((cache.Kc, cache.Kmax, k64), (cache.Vc, cache.Vmax, v64)):
                c = codes.cpu().numpy()[tab[np.arange(have[r]) // bs], :, np.arange(have[r]) % bs].astype(np.float64)
                held.append(c * (most.cpu().numpy()[tab[np.arange(have[r]) // bs]].astype(np.float64) / 127)[..., None])
                assert bool((np.abs(held[-1] - x[r, : have[r]]) <= off[len(held) - 1][..., None] * (1 + 1e-12)).all())
            for i in range(int(have[r] - add[r]), int(have[r])):
                for j in range(nh):
                    s = k64[r, : i + 1, j] @ q64[r, i, j] / d**0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o, A = p @ v64[r, : i + 1, j], p @ np.abs(v64[r, : i + 1, j])
                    e = np.abs(q64[r, i, j]).sum() * off[0][: i + 1, j].max() / d**0.5
                    dv = off[1][: i + 1, j].max()
                    E = (np.abs(k64[r, : i + 1, j]) @ np.abs(q64[r, i, j])).max() / d**0.5 + e
                    own = tolerance(np.abs(o) + A * np.expm1(2 * e) + dv, A * np.exp(2 * e) + dv, np.array(E), i + 1, 127 * 2 * dv)
                    bound = A * np.expm1(2 * e) + dv + own + BF16_TOL * np.abs(block).max()
                    assert bool((np.abs(got[at_row, j] - block[r, i, j]) <= bound).all())
                at_row += 1
    assert k > 15
