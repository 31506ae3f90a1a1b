"""GPU parity of the key/value cache in 8 bits against its float64 oracle.

Tables, slots and codes are whole numbers and equal.  Maxima are bf16 values and equal.

Attention, a row's output o = sum p v with A = sum p |v| (p the softmax weights): a weight is rounded to fp16,
2^-11 of itself; its score is off by at most 2^-19 of the largest scale sum |q k|, E (products of 11 and 8
bits are exact, at most 256 of them are added in fp32, the tensor cores' additions cut off instead of rounding),
and by a few 2^-24 of the exponent's terms, at most 2^-15 of a weight while they stay below 2^6; each of the two counts for a weight and
for the denominator, and o to half a bf16 step, 2^-8:
    |got - o| <= A (2^-11 + 2 E 2^-19 + 2 2^-15) + 2^-8 |o| + n 2^-35 M
The last term: n tokens' weights times their scales, p' in the kernel, are fp16 too, whose smallest half step is 2^-25, and the base that
they are taken from leaves the largest one of a row at 2^10 at least (the base moves to the largest less 10).  So the denominator,
the sum of p' / scale, is at least 2^10 / max scale, and n products of 2^-25 with a code of at most 127 come to n 2^-35 of the
largest value M that the request's blocks can hold, 127 times their largest scale.
"""
import numpy as np
import pytest
import torch

from oracle import kv_cache_oracle as kvo
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from gpu_harness import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


def _status_ok():
    torch.cuda.synchronize()
    assert mlp.mlp_sync_status() == mlp.MLP_OK, mlp.last_error()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------------------------------------ block tables
class Plan:
    def __init__(self, add, lens, width, bs, n_free, taken, rows, seed=0):
        rng = np.random.default_rng(seed)
        n = len(add)
        self.bs, self.rows = bs, rows
        self.add, self.lens = np.asarray(add, np.int32), np.asarray(lens, np.int32)
        self.table = rng.integers(-5, 5000, (n, width)).astype(np.int32)
        self.free = rng.permutation(100000)[:n_free].astype(np.int32)
        self.taken = taken
        self.dev = {k: i32(getattr(self, k)) for k in ("add", "lens", "table", "free")}
        self.dev["taken"] = i32([taken])
        self.out = {k: torch.full((m,), 77, dtype=torch.int32, device="cuda")
                    for k, m in (("lens", n), ("taken", 1), ("cu", n + 1), ("pos", rows), ("slots", rows), ("status", 1))}

    def run(self, stream=None):
        d, o = self.dev, self.out
        mlp.kv_plan(d["add"], d["lens"], d["table"], d["free"], d["taken"], self.bs, o["lens"], o["taken"], o["cu"], o["pos"],
                    o["slots"], o["status"], stream=stream)

    def check(self):
        status, lens, taken, cu, pos, slots, table = kvo.plan(self.add, self.lens, self.table, self.free, self.taken, self.bs, self.rows)
        o = {k: v.cpu().numpy() for k, v in self.out.items()}
        assert o["status"][0] == status and o["taken"][0] == taken
        for name, want in (("lens", lens), ("cu", cu), ("pos", pos), ("slots", slots)):
            np.testing.assert_array_equal(o[name], want, err_msg=name)
        np.testing.assert_array_equal(self.dev["table"].cpu().numpy(), table)
        return status


PLANS = [  # requests, new tokens up to, held up to, bs, padded rows
    (1, 1, 0, 16, 0), (1, 1, 16, 16, 5), (3, 0, 40, 32, 1), (64, 1, 300, 16, 0), (31, 70, 0, 64, 9), (257, 40, 500, 32, 0),
    (1000, 3, 90, 16, 100), (4096, 1, 33, 16, 0), (5, 3000, 100, 64, 2000)]


@pytest.mark.parametrize("n,most,held,bs,pad", PLANS)
def test_plan(n, most, held, bs, pad):
    rng = np.random.default_rng(n + most)
    add, lens = rng.integers(0, most + 1, n), rng.integers(0, held + 1, n)
    width = int((add + lens).max() + bs - 1) // bs + 1
    need = int(((lens + add + bs - 1) // bs - (lens + bs - 1) // bs).sum())
    p = Plan(add, lens, width, bs, need + 3, 3, int(add.sum()) + pad + (add.sum() + pad == 0))  # every free block is taken
    p.run()
    _status_ok()
    assert p.check() == 0


@pytest.mark.parametrize("change,bit", [(dict(n_free=12), 1), (dict(taken=-1), 1), (dict(width=4), 2), (dict(rows=99), 4),
                                        (dict(add=[50, -1, 51]), 8), (dict(lens=[16, 7, -3]), 8), (dict(rows=99, n_free=12), 5)])
def test_plan_refuses_a_step_whole(change, bit):
    a = dict(add=[50, 0, 50], lens=[16, 7, 15], width=5, bs=16, n_free=13, taken=5, rows=100)
    ok = Plan(**a)
    ok.run()
    p = Plan(**(a | change))
    p.run()
    _status_ok()
    assert ok.check() == 0
    assert p.check() & bit


def test_plan_with_entries_that_are_no_blocks():
    """A partly filled block's entry that is no block gives a slot outside every pool, never one that wrapped round."""
    p = Plan([3, 3, 3, 3], [1, 1, 1, 1], 2, 16, 9, 0, 12)
    p.table[:, 0] = [2**31 - 1, -(2**31), 1 << 28, -1]
    p.dev["table"] = i32(p.table)
    p.run()
    _status_ok()
    assert p.check() == 0
    assert bool((p.out["slots"] < 0).all())


def test_plan_with_lengths_near_the_largest():
    """Sums that pass 32 bits are refused, not wrapped round."""
    p = Plan([2**31 - 1] * 5, [2**31 - 1] * 5, 8, 64, 100, 0, 70)
    p.run()
    _status_ok()
    assert p.check() == 7


# ------------------------------------------------------------------------------------------ the write
class Pool:
    def __init__(self, blocks, nk, bs, d, seed=0):
        rng = np.random.default_rng(seed)
        self.shape = (blocks, nk, bs, d)
        self.Kc, self.Vc = (rng.integers(-127, 128, self.shape).astype(np.int8) for _ in range(2))
        self.Kmax, self.Vmax = (to_f64(torch.from_numpy(np.exp(rng.normal(0, 1, (blocks, nk)))).to(torch.bfloat16)).astype(np.float32)
                                for _ in range(2))
        self.dev = [torch.from_numpy(x).cuda() for x in (self.Kc, self.Vc, self.Kmax, self.Vmax)]


def _rows(T, nk, d, gap, seed, spread=1.0):
    """[T, nk, d] rows of a wider buffer."""
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(T, nk * d + gap, generator=g) * spread).to(torch.bfloat16).cuda()
    return flat[:, : nk * d].view(T, nk, d)


def check_write(pool, K, V, slots):
    got = [t.cpu().numpy() for t in pool.dev]
    for x, c, m, gc, gm in ((K, pool.Kc, pool.Kmax, got[0], got[2]), (V, pool.Vc, pool.Vmax, got[1], got[3])):
        codes, most = kvo.write(to_f64(x.cpu()), slots, c, m)
        np.testing.assert_array_equal(gm.astype(np.float64), most)
        np.testing.assert_array_equal(gc, codes)


WRITES = [  # heads, d, bs, gap, runs (block, place, tokens); None: a row without a slot
    (1, 32, 16, 0, [(3, 0, 1)]),
    (2, 64, 16, 8, [(3, 15, 1), None, (0, 0, 16), (5, 4, 12), (1, 7, 3)]),
    (8, 128, 32, 0, [(b, b % 32, 1) for b in range(20)] + [None]),
    (3, 96, 64, 16, [(2, 0, 64), (4, 0, 64), (1, 60, 4), (0, 0, 33), None, None]),
    (4, 160, 16, 24, [(b, 0, 16) for b in range(40)] + [(40, 0, 5)]),
    (2, 224, 32, 0, [(1, 31, 1), (2, 0, 32), (0, 17, 2)]),
    (2, 192, 64, 8, [(1, 63, 1), (2, 0, 50), (0, 17, 20)]),
    (5, 256, 64, 0, [(1, 33, 31), (2, 0, 64), (0, 0, 1)]),
]


def _slots(runs, bs):
    return np.array([s for r in runs for s in ([-1] if r is None else range(r[0] * bs + r[1], r[0] * bs + r[1] + r[2]))], np.int32)


@pytest.mark.parametrize("spread", [0.01, 1.0, 100.0])  # maxima that stay, that grow now and then, that all grow
@pytest.mark.parametrize("nk,d,bs,gap,runs", WRITES)
def test_write(nk, d, bs, gap, runs, spread):
    pool = Pool(45, nk, bs, d)
    slots = _slots(runs, bs)
    K, V = _rows(len(slots), nk, d, gap, 1, spread), _rows(len(slots), nk, d, gap, 2, spread)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


def test_write_many_tokens_and_heads():
    """The launch that looks through 16 tokens a CTA: ragged prompts that begin anywhere in it, single tokens between them."""
    rng = np.random.default_rng(5)
    runs, block = [], 0
    while block < 290:
        n = int(rng.integers(1, 90))
        off = int(rng.integers(0, 16)) if n < 5 else 0
        while n > 0:
            runs.append((block, off, min(n, 16 - off)))
            n -= min(n, 16 - off)
            block, off = block + 1, 0
        if rng.random() < 0.3:
            runs.append(None)
    pool = Pool(300, 6, 16, 64)
    slots = _slots(runs, 16)
    K, V = _rows(len(slots), 6, 64, 0, 1), _rows(len(slots), 6, 64, 0, 2)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


def test_write_ties_zeros_tiny_and_not_finite():
    """Codes that are ties go to even; a block of zeros, one below 2^-80, one with an infinity, one with a NaN, and one that
    held a NaN before."""
    pool = Pool(7, 1, 16, 32)
    pool.Kmax[5] = float("nan")
    pool.dev[2][5] = float("nan")
    slots = _slots([(0, 0, 2), (1, 0, 16), (2, 3, 1), (3, 0, 4), (4, 2, 3), (5, 4, 1), (6, 0, 1)], 16)
    K = torch.zeros(len(slots), 1, 32)
    K[0, 0] = torch.arange(32) * 2.0 + 1  # of 254: half codes, all exact in bf16
    K[1, 0, 0] = 254.0
    K[18, 0, :] = float("inf")
    K[19, 0, 5] = float("-inf")
    K[23, 0, 31] = float("nan")
    K[27, 0] = torch.linspace(-3, 3, 32) * 2.0**-110
    V = K.flip(-1)
    K, V = K.to(torch.bfloat16).cuda(), V.to(torch.bfloat16).cuda()
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


def test_write_leaves_out_slots_that_are_not_there():
    pool = Pool(3, 2, 16, 32)
    slots = np.array([48, 5, -7, 2**31 - 1, 47, -(2**31), 49], np.int32)
    K, V = _rows(7, 2, 32, 0, 1), _rows(7, 2, 32, 0, 2)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


# ------------------------------------------------------------------------------------------ the attention
def tolerance(o, A, E, n, M):
    return A * (2.0**-11 + 2 * E[..., None] * 2.0**-19 + 2 * 2.0**-15) + 2.0**-8 * np.abs(o) + n * 2.0**-35 * M


def largest(most, table, length, bs):
    """The largest value that the blocks of a request's tokens can hold."""
    blocks = [int(b) for b in table[: -(-max(length, 0) // bs)] if 0 <= b < len(most)]
    return float(np.max(most[blocks])) if blocks else 0.0


class Attn:
    """Requests of lens tokens with new[r] rows each (0 for none), their blocks anywhere in a pool."""

    def __init__(self, lens, new, nq, nk, d, bs, pad=0, gap=0, qscale=1.0, seed=0, width=None, spare=2, scale=None):
        rng = np.random.default_rng(seed)
        n = len(lens)
        self.lens, self.new = np.asarray(lens), np.asarray(new)
        have = -(-self.lens // bs)
        self.width = width or max(1, int(have.max()))
        blocks = int(have.sum()) + spare
        order = rng.permutation(blocks)
        self.table = np.full((n, self.width), -1, np.int32)
        at = 0
        for r in range(n):
            k = min(int(have[r]), self.width)
            self.table[r, :k] = order[at : at + k]
            at += k
        self.pool = Pool(blocks, nk, bs, d, seed + 1)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        T = int(self.cu[-1]) + pad
        self.Q = _rows(T, nq, d, gap, seed + 2, qscale)
        self.whole = torch.full((T + 1, nq * d + gap), 7.0, dtype=torch.bfloat16, device="cuda")
        self.O = self.whole[:T, : nq * d].view(T, nq, d)
        self.nq, self.nk, self.d, self.bs, self.T, self.gap, self.scale = nq, nk, d, bs, T, gap, scale
        self.args()

    def args(self):
        self.dt, self.dl, self.dc = i32(self.table), i32(self.lens), i32(self.cu)
        self.ws = torch.full((mlp.kv_attn_workspace(self.d),), float("nan"), device="cuda")

    def run(self, stream=None):
        mlp.kv_attn(self.Q, *self.pool.dev, self.dt, self.dl, self.dc, self.O, self.ws, scale=self.scale, stream=stream)

    def check(self):
        q, got = to_f64(self.Q.cpu()), to_f64(self.O.cpu())
        p = self.pool
        scale = float(np.float32(self.d**-0.5 if self.scale is None else self.scale))
        used, right = np.zeros(self.T, bool), np.zeros(got.shape, bool)  # a row that two requests claim may be either's
        for r in range(len(self.lens)):
            rows = slice(int(self.cu[r]), int(self.cu[r + 1]))
            if not 0 <= rows.start < rows.stop <= self.T:
                continue
            used[rows] = True
            o, A, E = kvo.attn(q[rows], p.Kc, p.Vc, p.Kmax, p.Vmax, self.table[r], int(self.lens[r]), scale)
            length = min(int(self.lens[r]), self.width * self.bs)
            right[rows] |= np.abs(got[rows] - o) <= tolerance(o, A, E, length, largest(p.Vmax, self.table[r], length, self.bs))
        wrong = np.argwhere(~right[used])
        assert len(wrong) == 0, (len(wrong), wrong[:5])
        w = self.whole.clone()
        w[: self.T, : self.nq * self.d][torch.from_numpy(used).cuda()] = 7
        assert bool(torch.all(w == 7)), "rows or gaps that belong to no request were written"


ATTNS = [  # lens, new, nq, nk, d, bs
    ([1], [1], 1, 1, 32, 16),
    ([16], [1], 4, 1, 64, 16),
    ([17, 0, 1], [1, 1, 1], 8, 2, 128, 16),
    ([15, 33, 64, 65, 200], [1, 1, 1, 1, 1], 6, 2, 96, 32),
    ([137, 5, 900], [1, 0, 1], 32, 8, 128, 64),
    ([300, 3], [5, 3], 16, 4, 160, 16),
    ([257, 100], [1, 7], 12, 4, 192, 32),
    ([130, 1000], [2, 1], 3, 1, 224, 64),
    ([77, 128], [4, 1], 10, 2, 256, 16),
    ([4, 2, 1], [6, 2, 3], 4, 4, 64, 16),             # rows of a request with fewer tokens than rows: they see none
    ([50, 60], [50, 37], 6, 2, 128, 16),              # a whole prompt, several tiles of rows
    ([5000], [1], 2, 1, 128, 16),                     # one request over many CTAs
    ([6000, 20, 1, 3000], [1, 1, 1, 1], 24, 3, 64, 32),
    ([2500], [3], 40, 1, 32, 64),
    (list(range(0, 150)), [1] * 150, 4, 2, 32, 16),
]


@pytest.mark.parametrize("pad,gap", [(0, 0), (3, 8)])
@pytest.mark.parametrize("lens,new,nq,nk,d,bs", ATTNS)
def test_attn(lens, new, nq, nk, d, bs, pad, gap):
    c = Attn(lens, new, nq, nk, d, bs, pad, gap)
    c.run()
    _status_ok()
    c.check()


def test_attn_more_requests_than_threads():
    rng = np.random.default_rng(3)
    c = Attn(rng.integers(0, 40, 1500), rng.integers(0, 3, 1500), 2, 1, 32, 16, pad=1)
    c.run()
    _status_ok()
    c.check()


def test_attn_twice_is_the_same_and_on_another_stream():
    c = Attn([4000, 333, 1], [1, 2, 1], 16, 4, 128, 16)
    c.run()
    _status_ok()
    first = c.O.clone()
    c.check()
    c.O.fill_(7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(first, c.O)


@pytest.mark.parametrize("qscale,scale", [(1e-30, None), (30.0, 0.02), (1e-3, 5.0), (200.0, 0.0005)])
def test_attn_queries_of_any_size(qscale, scale):
    c = Attn([100, 700], [1, 1], 8, 2, 128, 16, qscale=qscale, scale=scale)
    c.run()
    _status_ok()
    c.check()


def test_attn_a_sharp_softmax():
    """Scores spread over hundreds: one token carries nearly all, and the maximum grows along the way."""
    c = Attn([1000], [1], 4, 1, 64, 16, qscale=8.0, scale=1.0)
    c.pool.Kmax[:] = 1.0
    c.pool.dev[2].fill_(1.0)
    c.run()
    _status_ok()
    c.check()


def test_attn_value_maxima_far_apart():
    """Blocks whose values differ by 2^40 in scale, and blocks of zeros: what a small weight times a large value gives counts as
    in the formula."""
    c = Attn([640, 200], [1, 1], 8, 2, 64, 16, qscale=3.0)
    rng = np.random.default_rng(1)
    v = np.exp2(rng.integers(-20, 21, c.pool.Vmax.shape)).astype(np.float32)
    v[::7] = 0
    c.pool.Vmax[:] = v
    c.pool.dev[3].copy_(torch.from_numpy(v))
    c.run()
    _status_ok()
    c.check()


@pytest.mark.parametrize("most", [2.0**-79, 2.0**100])
def test_attn_values_of_any_size(most):
    """Values all tiny or all huge, over a long request: neither the sums nor the denominator leave fp32's range.  The
    output is of the values' size, so the bound is."""
    c = Attn([3000, 40], [1, 1], 8, 2, 64, 16)
    c.pool.Vmax[:] = most
    c.pool.dev[3].fill_(most)
    c.run()
    _status_ok()
    c.check()


def test_attn_a_block_of_zeros_that_carries_the_weight():
    """The block with by far the largest scores holds values of zero (their maximum 0, their codes 0): its weight counts in the
    denominator beside blocks of values 2^20 times and 2^-60 times as large as usual."""
    for scale in (2.0**20, 1.0, 2.0**-60):
        c = Attn([200], [1], 4, 1, 64, 16, qscale=4.0)
        zero = int(c.table[0, 5])
        c.pool.Vmax[:] = scale
        c.pool.Vmax[zero], c.pool.Vc[zero] = 0, 0
        c.pool.Kmax[:], c.pool.Kmax[zero] = 1.0, 3.0
        c.pool.dev = [torch.from_numpy(x).cuda() for x in (c.pool.Kc, c.pool.Vc, c.pool.Kmax, c.pool.Vmax)]
        c.run()
        _status_ok()
        c.check()


def test_attn_what_is_not_seen_does_not_count():
    """Blocks behind a request's tokens, and blocks of another one, full of NaN; tables with rubbish behind the request's blocks;
    a table entry outside the pool, whose tokens are left out; codes behind the last token."""
    c = Attn([70, 33, 20, 0], [1, 2, 4, 1], 8, 2, 128, 16, width=9, spare=4)
    used = {int(b) for r in range(4) for b in c.table[r, : -(-int(c.lens[r]) // 16)]}
    for b in set(range(c.pool.shape[0])) - used:
        for i in (2, 3):
            c.pool.dev[i][b] = float("nan")
    for r in range(4):
        c.table[r, -(-int(c.lens[r]) // 16) :] = [2**31 - 1, -1, -(2**31)][r % 3]
    c.table[0, 2] = c.pool.shape[0]
    c.table[1, 0] = -1
    c.args()
    c.run()
    _status_ok()
    c.check()


def test_attn_a_block_of_nan_reaches_the_rows_that_see_it():
    """The second row sees the block that begins with its own token, the first does not."""
    c = Attn([33], [2], 4, 2, 64, 16)
    bad = int(c.table[0, 2])
    for i in (2, 3):
        c.pool.dev[i][bad, 1] = float("nan")
    c.run()
    _status_ok()
    assert torch.isnan(c.O[1, 2:]).all()
    c.pool.Kmax[bad], c.pool.Vmax[bad] = 1, 1
    clean = c.O.clone()
    c.pool.dev[2][bad], c.pool.dev[3][bad] = 1, 1
    c.run()
    _status_ok()
    c.check()
    assert torch.equal(clean[0], c.O[0])


def test_attn_a_query_that_is_not_finite_keeps_to_its_row():
    c = Attn([90, 40], [2, 1], 4, 2, 64, 16)
    c.run()
    clean = c.O.clone()
    c.Q[1, 2, 5] = float("nan")
    c.Q[2, 0, 1] = float("inf")
    c.run()
    _status_ok()
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    assert torch.equal(c.O[~bad], clean[~bad])
    assert torch.isnan(c.O[1, 2]).all()


@pytest.mark.parametrize("lens,cu", [([40, 40, 40], [0, 1, 1, 2]), ([40, 40, 40], [0, 3, 1, 2]), ([40, 40, 40], [0, 1, 9, 2]),
                                     ([40, -5, 40], [0, 1, 2, 3]), ([2**31 - 1, 40, 40], [0, 1, 2, 3]), ([40, 40, 40], [-1, 1, 2, 3])])
def test_attn_lengths_and_offsets_that_are_wrong(lens, cu):
    """Requests whose offsets are no range of rows are left out, negative lengths hold nothing, lengths behind the table's
    end are cut off there."""
    c = Attn([40, 40, 40], [1, 1, 1], 4, 1, 64, 16)
    c.lens, c.cu = np.asarray(lens), np.asarray(cu, np.int32)
    c.args()
    c.run()
    _status_ok()
    c.check()


def test_cache_beyond_32_bit_offsets():
    """Slots of the last blocks of a pool whose codes take over 4 GB."""
    nk, d, bs = 64, 256, 64
    blocks = (1 << 32) // (nk * bs * d) + 3
    cache = mlp.KVCache(blocks, nk, bs, d)
    T = 70
    K, V = _rows(T, nk, d, 0, 1), _rows(T, nk, d, 0, 2)
    table = np.array([[blocks - 1, blocks - 2]], np.int32)
    slots = np.array([int(table[0, j // bs]) * bs + j % bs for j in range(T)], np.int32)
    mlp.kv_write(K, V, i32(slots), cache.Kc, cache.Vc, cache.Kmax, cache.Vmax)
    Q, O = _rows(1, nk, d, 0, 3), torch.zeros(1, nk, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mlp.kv_attn_workspace(d), device="cuda")
    mlp.kv_attn(Q, cache.Kc, cache.Vc, cache.Kmax, cache.Vmax, i32(table), i32([T]), i32([0, 1]), O, ws)
    _status_ok()
    assert int(cache.Kc[:-2].count_nonzero()) == 0
    held = [x[-2:].cpu().numpy() for x in (cache.Kc, cache.Vc, cache.Kmax, cache.Vmax)]
    for x, codes, most in ((K, held[0], held[2]), (V, held[1], held[3])):
        want = kvo.write(to_f64(x.cpu()), slots - (blocks - 2) * bs, np.zeros_like(codes), np.zeros_like(most))
        np.testing.assert_array_equal(codes, want[0])
        np.testing.assert_array_equal(most.astype(np.float64), want[1])
    o, A, E = kvo.attn(to_f64(Q.cpu()), *held, table[0] - (blocks - 2), T, float(np.float32(d**-0.5)))
    assert bool((np.abs(to_f64(O.cpu()) - o) <= tolerance(o, A, E, T, held[3].max())).all())


# ------------------------------------------------------------------------------------------ a step of a serving loop
class Loop:
    """A layer's cache as a serving loop uses it: prompts, then single tokens and drafts, every step by the same calls.  The
    queries' and keys' norm and rotation come before the write; a float64 copy of what was written is kept apart."""

    def __init__(self, n, nq, nk, d, bs, width, blocks, rows, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.nq, self.nk, self.d, self.bs, self.rows = n, nq, nk, d, bs, rows
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cache = mlp.KVCache(blocks, nk, bs, d)
        self.table, self.free = torch.full((n, width), -1, dtype=torch.int32, device="cuda"), torch.randperm(blocks, generator=g).int().cuda()
        self.add, self.lens, self.taken = z(n), [z(n), z(n)], [z(1), z(1)]
        self.cu, self.pos, self.slots, self.status = z(n + 1), z(rows), z(rows), z(1)
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.QKV, self.Qr, self.Kr, self.O = bf(rows, (nq + 2 * nk) * d), bf(rows, nq, d), bf(rows, nk, d), bf(rows, nq, d)
        self.Q, self.K = self.QKV[:, : nq * d].view(rows, nq, d), self.QKV[:, nq * d : (nq + nk) * d].view(rows, nk, d)
        self.V = self.QKV[:, (nq + nk) * d :].view(rows, nk, d)
        self.inv = (10000.0 ** -torch.linspace(0, 1, d // 2, dtype=torch.float64)).float().cuda()
        self.wq, self.wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
        self.ws = torch.empty(mlp.kv_attn_workspace(d), device="cuda")

    def step(self, k):
        """Step k: k % 2 says which array of lengths is the older one."""
        a, b = k % 2, 1 - k % 2
        mlp.kv_plan(self.add, self.lens[a], self.table, self.free, self.taken[a], self.bs, self.lens[b], self.taken[b], self.cu,
                    self.pos, self.slots, self.status)
        mlp.qk_norm_rope_fwd(self.Q, self.K, self.Qr, self.Kr, self.pos[None], self.inv, wq=self.wq, wk=self.wk)
        c = self.cache
        mlp.kv_write(self.Kr, self.V, self.slots, c.Kc, c.Vc, c.Kmax, c.Vmax)
        mlp.kv_attn(self.Qr, c.Kc, c.Vc, c.Kmax, c.Vmax, self.table, self.lens[b], self.cu, self.O, self.ws)


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    """Prompts, single tokens, drafts, a request that rests, a batch with padded rows; captured as two graphs that take turns."""
    n, nq, nk, d, bs, rows = 4, 8, 2, 128, 16, 64
    L = Loop(n, nq, nk, d, bs, width=8, blocks=40, rows=rows)
    graphs = []
    if captured:
        for k in (0, 1):
            L.step(k)  # first calls outside a capture, with nothing to add
        torch.cuda.synchronize()
        for k in (0, 1):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                L.step(k)
            graphs.append(graph)
    g = torch.Generator().manual_seed(9)
    lens = np.zeros(n, np.int32)
    table, taken = L.table.cpu().numpy(), 0
    codes = [np.zeros((40, nk, bs, d), np.int8) for _ in range(2)]
    most = [np.zeros((40, nk)) for _ in range(2)]
    for k, add in enumerate([[20, 1, 0, 40], [1, 1, 33, 1], [1, 1, 1, 1], [3, 0, 5, 1], [1, 1, 1, 1], [1, 1, 1, 1], [14, 1, 1, 1]]):
        add = np.array(add, np.int32)
        L.add.copy_(torch.from_numpy(add))
        L.QKV.copy_((torch.randn(L.QKV.shape, generator=g) * (1 + 0.2 * k)).to(torch.bfloat16))
        L.O.fill_(7.0)
        if captured:
            graphs[k % 2].replay()
        else:
            L.step(k)
        _status_ok()
        status, lens, taken, cu, pos, slots, table = kvo.plan(add, lens, table, L.free.cpu().numpy(), taken, bs, rows)
        assert status == 0 and int(L.status) == 0
        np.testing.assert_array_equal(L.slots.cpu().numpy(), slots)
        np.testing.assert_array_equal(L.lens[1 - k % 2].cpu().numpy(), lens)
        np.testing.assert_array_equal(L.pos.cpu().numpy(), pos)
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


def test_two_captured_attentions_at_once():
    """Two graphs with a workspace each, replayed on two streams at once, give what their calls alone give."""
    cases = [Attn([3000, 500], [1, 1], 8, 2, 128, 16, seed=1), Attn([100, 2500], [2, 1], 8, 2, 128, 16, seed=5)]
    want, graphs = [], []
    for c in cases:
        c.run()
        _status_ok()
        want.append(c.O.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c in cases:
            c.O.fill_(7.0)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.O, w)


@pytest.mark.parametrize("bs,nk,d", [(64, 64, 32), (32, 48, 96), (16, 40, 128), (64, 20, 160)])
def test_write_many_heads(bs, nk, d):
    """So many heads that a CTA takes a block's tokens and several heads: whole blocks, parts of them, runs of a few tokens and
    single ones in any order, at any place of the CTA's tokens, over codes that move."""
    rng = np.random.default_rng(bs + nk)
    runs, block = [], 0
    while sum(1 if r is None else r[2] for r in runs) < 420:
        off = int(rng.integers(0, bs))
        n = int(rng.choice([1, 1, 2, 5, bs]))
        if n == bs:
            off = int(rng.choice([0, off]))
        runs.append((block, off, min(n, bs - off)))
        block += 1
        if rng.random() < 0.1:
            runs.append(None)
    order = rng.permutation(block)
    runs = [r if r is None else (int(order[r[0]]), r[1], r[2]) for r in runs]
    pool = Pool(block, nk, bs, d)
    slots = _slots(runs, bs)
    K, V = _rows(len(slots), nk, d, 16, 1), _rows(len(slots), nk, d, 0, 2, 2.0)
    mlp.kv_write(K, V, i32(slots), *pool.dev)
    _status_ok()
    check_write(pool, K, V, slots)


def test_calls_from_two_threads_on_two_streams():
    """Each thread's writes and attention on a stream and a cache of its own give what they give alone."""
    import threading

    def work(seed, stream, out):
        with torch.cuda.stream(stream):
            c = Attn([700, 33], [1, 2], 8, 2, 96, 16, seed=seed)
            slots = _slots([(0, 0, 16), (1, 0, 3)], 16)
            K, V = _rows(19, 2, 96, 0, seed), _rows(19, 2, 96, 0, seed + 1)
            for _ in range(20):
                mlp.kv_write(K, V, i32(slots), *c.pool.dev)
                c.run()
            stream.synchronize()
            out.append((c.O.clone(), [t.clone() for t in c.pool.dev]))

    alone, both = [[], []], [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        work(50 + 10 * k, streams[k], alone[k])
    threads = [threading.Thread(target=work, args=(50 + 10 * k, streams[k], both[k])) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _status_ok()
    for a, b in zip(alone, both):
        assert torch.equal(a[0][0], b[0][0]) and all(torch.equal(x, y) for x, y in zip(a[0][1], b[0][1]))


@pytest.mark.parametrize("group,new", [(5, 1), (16, 1), (7, 3), (10, 4)])  # tiles of 8, 16 and 24 rows, one to three of them
@pytest.mark.parametrize("d", range(32, 257, 32))
def test_attn_every_head_size_and_tile(d, group, new):
    """Requests over several CTAs and short ones, in every kernel that there is."""
    c = Attn([1500, new, 90, 16], [new, new, new, new], 2 * group, 2, d, 16, pad=2, gap=8, seed=d + group)
    c.run()
    _status_ok()
    c.check()


def test_attn_as_many_requests_as_there_may_be():
    c = Attn([3] * 4096, [1] * 4096, 1, 1, 32, 16, seed=2)
    c.run()
    _status_ok()
    c.check()
