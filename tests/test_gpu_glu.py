"""GPU parity of the gated feed-forward block against the float64 oracle.

Every stage is compared from the bf16 tensors that the stage before stored, so each
bound is that stage's own:
  * a product of n terms accumulated in fp32 is off by at most n steps of 2^-23 of
    the sum of the terms' magnitudes (each addition keeps 24 bits, rounded any way);
  * the gate and its slope are off by 2^-17 relative: exp and reciprocal approximations
    are good to 2^-21, and exp's argument (at most 80) carries a rounding of 2^-24 relative;
  * a value stored as bf16 is off by half a step, 2^-8 of it.
These bounds hold element by element.  In the 2-norm the whole error of a bf16 output
stays under 2^-8 of the result, the most its last rounding alone can make, and of an
fp32 output under n 2^-24 (measured for these GEMMs: 2.3e-6 at n = 2048).
"""
import numpy as np
import pytest
import torch

from oracle import glu_oracle as glo
from oracle import mlp_oracle
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from gpu_harness import to_f64

pytestmark = pytest.mark.gpu

ACT = {"silu": mlp.GLU_SILU, "gelu": mlp.GLU_GELU}
SEED, OFFSET = 1234, 77


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


@pytest.fixture
def cta_pair_mode(request):
    mlp.mlp_set_cta_pair(request.param)
    yield request.param
    mlp.mlp_set_cta_pair(-1)


def _status_ok():
    torch.cuda.synchronize()
    assert mlp.mlp_sync_status() == mlp.MLP_OK, mlp.last_error()


def _guarded(rows, cols, dtype=torch.bfloat16):
    """A [rows, cols] tensor of NaN with 40 more rows of 7 behind it: (view, those rows)."""
    whole = torch.full((rows + 40, cols), float("nan"), dtype=dtype, device="cuda")
    whole[rows:] = 7
    return whole[:rows], whole[rows:]


class Case:
    def __init__(self, T, h, ffn, act="silu", p=0.1, bias=True, seed=0, std=None):
        g = torch.Generator().manual_seed(seed)
        std = std or 1.0 / np.sqrt(h)
        r = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(torch.bfloat16).cuda()  # noqa: E731
        self.T, self.h, self.ffn, self.act, self.p = T, h, ffn, act, p
        self.X, self.A, self.B, self.dO = r(T, h), r(h, 2 * ffn, k=std), r(ffn, h, k=1.0 / np.sqrt(ffn)), r(T, h)
        self.a, self.b = (r(2 * ffn), r(h)) if bias else (None, None)

    def fwd(self, GU, Y, O, R=None, stream=None, t=1):
        mlp.glu_fwd(self.h, self.ffn, t, self.T, self.p, SEED, OFFSET, ACT[self.act], self.X, self.A, self.a, self.B, self.b,
                    R, GU, Y, O, stream)

    def bwd_input(self, GU, dZ, dGU, dX, residual_grad=1, stream=None):
        mlp.glu_bwd_input(self.h, self.ffn, 1, self.T, self.p, SEED, OFFSET, ACT[self.act], residual_grad, self.dO, self.A,
                          self.B, GU, dZ, dGU, dX, stream)

    def bwd_weights(self, dZ, Y, dGU, dA, da, dB, db, scratch=None, accumulate=0, stream=None):
        mlp.glu_bwd_weights(self.h, self.ffn, 1, self.T, accumulate, self.X, dZ, Y, dGU, dA, da, dB, db, scratch, stream)


def f64(t):
    return None if t is None else to_f64(t)


def _check(got, ref, bound, what, norm_bar):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    over = err - bound
    assert over.max() <= 0, (what, err.flat[over.argmax()], bound.flat[over.argmax()], np.unravel_index(over.argmax(), over.shape))
    assert np.linalg.norm(got - ref) <= norm_bar * np.linalg.norm(ref), (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))


BF = 2.0**-8
NORM = 2.0**-8


def _acc(x, w, n):
    return n * 2.0**-23 * (np.abs(x) @ np.abs(w))


def _slope_max():
    return 1.13  # of both gates


def check_forward(c, GU, Y, O, R=None):
    X, A, a, B, b = (f64(x) for x in (c.X, c.A, c.a, c.B, c.b))
    ref = glo.gates(X, A, a)
    e = _acc(X, A, c.h) + 2.0**-23 * np.abs(ref)
    if GU is not None:
        _check(f64(GU), ref, BF * (np.abs(ref) + e) + e, "GU", NORM)
    y = glo.gated(ref, c.act)
    G, U = ref[:, :c.ffn], ref[:, c.ffn:]
    ey = _slope_max() * e[:, :c.ffn] * (np.abs(U) + e[:, c.ffn:]) + np.abs(glo.act(G, c.act)) * e[:, c.ffn:] + 2.0**-17 * np.abs(y)
    _check(f64(Y), y, BF * (np.abs(y) + ey) + ey, "Y", NORM)
    Ys, Rs = f64(Y), X if R is None else f64(R)
    o = glo.out(Ys, B, b, Rs, c.p, SEED, OFFSET)
    scale = glo.dropout_scale(c.p)
    eo = scale * (_acc(Ys, B, c.ffn) + 2.0**-22 * np.abs((o - Rs) / scale)) + 2.0**-23 * np.abs(o)
    _check(f64(O), o, BF * (np.abs(o) + eo) + eo, "O", NORM)


def check_backward_input(c, GU, dZ, dGU, dX, residual_grad=1):
    A, B, dO = f64(c.A), f64(c.B), f64(c.dO)
    z = glo.d_out(dO, c.p, SEED, OFFSET)
    if c.p > 0:
        _check(f64(dZ), z, BF * np.abs(z) * (1 + 2.0**-20) + 2.0**-22 * np.abs(z), "dZ", NORM)
    zs, gu = f64(dZ) if c.p > 0 else dO, f64(GU)
    ref = glo.d_gates(zs, B, gu, c.act)
    G, U = gu[:, :c.ffn], gu[:, c.ffn:]
    ea = _acc(zs, B.T, c.h)
    factor = np.concatenate([np.abs(U) * _slope_max(), np.abs(glo.act(G, c.act))], axis=1)
    # the slope is a difference of terms of size one near its zero: an absolute error of 2^-17
    dy = np.abs(zs @ B.T)
    e = np.concatenate([ea, ea], axis=1) * factor + 2.0**-17 * np.concatenate([dy * np.abs(U) * _slope_max(), np.abs(ref[:, c.ffn:])], axis=1)
    _check(f64(dGU), ref, BF * (np.abs(ref) + e) + e, "dGU", NORM)
    d = f64(dGU)
    ref = glo.d_input(d, A, dO if residual_grad else None)
    e = _acc(d, A.T, 2 * c.ffn) + 2.0**-23 * np.abs(ref)
    _check(f64(dX), ref, BF * (np.abs(ref) + e) + e, "dX", NORM)


def check_weights(c, dZ, Y, dGU, grads, before=None):
    X, z, y, d = f64(c.X), f64(dZ), f64(Y), f64(dGU)
    refs = glo.d_weights(X, z, y, d)
    one = np.ones((c.T, 1))
    bounds = (_acc(X.T, d, c.T), _acc(one.T, d, c.T)[0], _acc(y.T, z, c.T), _acc(one.T, z, c.T)[0])
    for k, (name, ref, e) in enumerate(zip(("dA", "da", "dB", "db"), refs, bounds)):
        if grads[k] is None:
            continue
        old = 0.0 if before is None else f64(before[k])
        ref = ref + old
        _check(f64(grads[k]), ref, e + 2.0**-22 * (np.abs(ref) + np.abs(old)) + 1e-30, name, max(c.T, 8) * 2.0**-24 + 2.0**-20)


SHAPES = [
    # T, h, ffn, act, p, bias: one token to a few tiles; sizes of every remainder that the layout allows
    (1, 8, 8, "silu", 0.0, False),
    (1, 256, 1024, "silu", 0.1, True),
    (2, 1024, 136, "gelu", 0.0, True),
    (5, 72, 264, "gelu", 0.5, True),
    (16, 2048, 640, "silu", 0.0, False),
    (17, 1032, 520, "silu", 0.1, True),
    (33, 520, 2744, "gelu", 0.1, False),
    (64, 1288, 384, "silu", 0.0, True),
    (65, 264, 72, "gelu", 0.1, True),
    (128, 1024, 1024, "silu", 0.1, True),
    (129, 1096, 200, "gelu", 0.0, False),
    (200, 320, 1000, "silu", 0.1, True),
    (257, 1032, 2744, "gelu", 0.1, True),
    (640, 2056, 328, "silu", 0.0, True),
    (1100, 264, 520, "gelu", 0.1, True),     # weight gradients of few tiles and a long reduction
    (1610, 136, 264, "silu", 0.0, True),
    (385, 3080, 264, "gelu", 0.1, False),
    # weights too large for the few-token launches: tiles of 256 x 256, shared out or not
    (300, 2056, 6152, "silu", 0.1, True),
    (1300, 2568, 1288, "gelu", 0.0, False),
    (2100, 520, 4104, "silu", 0.1, True),
]


@pytest.mark.parametrize("T,h,ffn,act,p,bias", SHAPES)
def test_forward_and_backward(T, h, ffn, act, p, bias):
    c = Case(T, h, ffn, act, p, bias)
    GU, g0 = _guarded(T, 2 * ffn)
    Y, g1 = _guarded(T, ffn)
    O, g2 = _guarded(T, h)
    c.fwd(GU, Y, O)
    _status_ok()
    check_forward(c, GU, Y, O)
    dZ, g3 = _guarded(T, h)
    dGU, g4 = _guarded(T, 2 * ffn)
    dX, g5 = _guarded(T, h)
    c.bwd_input(GU, dZ if p > 0 else None, dGU, dX)
    _status_ok()
    z = dZ if p > 0 else c.dO
    check_backward_input(c, GU, z, dGU, dX)
    f32 = torch.float32
    dA, g6 = _guarded(h, 2 * ffn, f32)
    dB, g7 = _guarded(ffn, h, f32)
    da = torch.full((2 * ffn,), float("nan"), device="cuda") if bias else None
    db = torch.full((h,), float("nan"), device="cuda") if bias else None
    c.bwd_weights(z, Y, dGU, dA, da, dB, db)
    _status_ok()
    check_weights(c, z, Y, dGU, (dA, da, dB, db))
    # and added to what is there
    before = [None if x is None else torch.randn(x.shape, device="cuda") for x in (dA, da, dB, db)]
    after = [None if x is None else x.clone() for x in before]
    c.bwd_weights(z, Y, dGU, *after, accumulate=1)
    _status_ok()
    check_weights(c, z, Y, dGU, after, before)
    for k, g in enumerate((g0, g1, g2, g3, g4, g5, g6, g7)):
        assert torch.all(g == 7), ("rows behind the last", k)


@pytest.mark.parametrize("cta_pair_mode", [0, 1], indirect=True, ids=["single", "pair"])
@pytest.mark.parametrize("T,h,ffn,act", [(300, 264, 392, "gelu"), (300, 1096, 392, "silu"), (100, 1096, 392, "gelu"),
                                          (700, 2568, 2056, "silu"), (530, 264, 136, "gelu")])
def test_both_cta_modes(T, h, ffn, act, cta_pair_mode):
    c = Case(T, h, ffn, act)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    GU, Y, O = torch.empty(T, 2 * ffn, **bf), torch.empty(T, ffn, **bf), torch.empty(T, h, **bf)
    c.fwd(GU, Y, O)
    dZ, dGU, dX = torch.empty(T, h, **bf), torch.empty(T, 2 * ffn, **bf), torch.empty(T, h, **bf)
    c.bwd_input(GU, dZ, dGU, dX)
    _status_ok()
    check_forward(c, GU, Y, O)
    check_backward_input(c, GU, dZ, dGU, dX)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_without_gates_stored_and_with_a_residual(T):
    """GU = NULL changes no bit of Y and O; R other than X is added; slices change nothing;
    the backward without the residual's gradient."""
    c = Case(T, 1032, 712, "silu")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    R = torch.randn(T, c.h, device="cuda").to(torch.bfloat16)
    GU = torch.empty(T, 2 * c.ffn, **bf)
    got = []
    for gu, t in ((GU, 1), (None, 1), (None, 89)):
        Y, O = torch.empty(T, c.ffn, **bf), torch.empty(T, c.h, **bf)
        c.fwd(gu, Y, O, R, t=t)
        got.append((Y, O))
    _status_ok()
    check_forward(c, GU, *got[0], R=R)
    for Y, O in got[1:]:
        assert torch.equal(Y, got[0][0]) and torch.equal(O, got[0][1])
    dZ, dGU, dX = torch.empty(T, c.h, **bf), torch.empty(T, 2 * c.ffn, **bf), torch.empty(T, c.h, **bf)
    c.bwd_input(GU, dZ, dGU, dX, residual_grad=0)
    _status_ok()
    check_backward_input(c, GU, dZ, dGU, dX, residual_grad=0)


@pytest.mark.parametrize("T,ffn,extra", [(1, 520, "bias"), (48, 520, "nothing"), (300, 520, "bias")])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_extreme_gates(T, ffn, extra, act):
    """Gates at the ends of the range: the gate's value and slope there are 0 or x and 0 or
    1; a NaN stays a NaN in its own row and reaches no other."""
    c = Case(T, 264, ffn, act, 0.0, True)
    c.a = torch.zeros_like(c.a)
    ends = torch.tensor([-3e38, -1e4, -100.0, -81.0, -30.5, 30.5, 90.0, 1e4], dtype=torch.bfloat16, device="cuda")
    c.A[:, :8] = 0
    c.a[:8] = ends
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if T > 1:
        c.X[T // 2, 3] = float("nan")
    GU, Y, O = torch.empty(T, 2 * ffn, **bf), torch.empty(T, ffn, **bf), torch.empty(T, c.h, **bf)
    c.fwd(GU, Y, O)
    dGU, dX = torch.empty(T, 2 * ffn, **bf), torch.empty(T, c.h, **bf)
    c.bwd_input(GU, None, dGU, dX)
    _status_ok()
    rows = [i for i in range(T) if T == 1 or i != T // 2]
    if T > 1:
        assert torch.isnan(Y[T // 2]).all() and torch.isnan(O[T // 2]).all()
        assert torch.isnan(dGU[T // 2]).all() and torch.isnan(dX[T // 2]).all()
    U = GU[rows, ffn:ffn + 8].float()
    dY = (c.dO.float() @ c.B.float().t())[rows, :8]
    y, dG, dU = Y[rows, :8].float(), dGU[rows, :8].float(), dGU[rows, ffn:ffn + 8].float()
    low, high = slice(0, 4), slice(5, 8)
    assert torch.all(y[:, low].abs() <= 1e-30) and torch.all(dG[:, low].abs() <= 1e-30) and torch.all(dU[:, low].abs() <= 1e-30)
    want = ends[high].float() * U[:, high]
    assert torch.all((y[:, high] - want).abs() <= 2.0**-7 * want.abs())
    # the product dY in fp32 differs from the kernel's by the order of its 264 terms
    slack = 264 * 2.0**-22 * (c.dO.float().abs() @ c.B.float().abs().t())[rows, :8]
    want = dY[:, high] * U[:, high]
    assert torch.all((dG[:, high] - want).abs() <= 2.0**-7 * want.abs() + slack[:, high] * U[:, high].abs() * 1.01)
    want = dY[:, high] * ends[high].float()
    assert torch.all((dU[:, high] - want).abs() <= 2.0**-7 * want.abs() + slack[:, high] * ends[high].float() * 1.01)


@pytest.mark.parametrize("T", [1, 27, 100, 600])
def test_graph_replay_streams_and_repeats_give_the_same_bits(T):
    """Eager calls on two streams at once, and two graphs captured on one stream and replayed at once:
    the bits of calls one after another; then new inputs under the same graph."""
    cs = [Case(T, 1096, 2744, "silu", 0.1, True, seed=s) for s in (1, 2)]
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def buffers(c):
        return dict(GU=torch.empty(T, 2 * c.ffn, **bf), Y=torch.empty(T, c.ffn, **bf), O=torch.empty(T, c.h, **bf),
                    dZ=torch.empty(T, c.h, **bf), dGU=torch.empty(T, 2 * c.ffn, **bf), dX=torch.empty(T, c.h, **bf),
                    dA=torch.empty(c.h, 2 * c.ffn, device="cuda"), da=torch.empty(2 * c.ffn, device="cuda"),
                    dB=torch.empty(c.ffn, c.h, device="cuda"), db=torch.empty(c.h, device="cuda"))

    def step(c, b):
        c.fwd(b["GU"], b["Y"], b["O"])
        c.bwd_input(b["GU"], b["dZ"], b["dGU"], b["dX"])
        c.bwd_weights(b["dZ"], b["Y"], b["dGU"], b["dA"], b["da"], b["dB"], b["db"])

    eager = [buffers(c) for c in cs]
    for c, b in zip(cs, eager):
        step(c, b)
    _status_ok()
    # eager on two streams at once
    streams = [torch.cuda.Stream() for _ in cs]
    again = [buffers(c) for c in cs]
    for s, c, b in zip(streams, cs, again):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                step(c, b)
    _status_ok()
    for b, r in zip(again, eager):
        for k in b:
            assert torch.equal(b[k], r[k]), ("two streams", k)
    # two graphs captured on one stream, replayed at once
    graphs, bufs = [], [buffers(c) for c in cs]
    one = torch.cuda.Stream()
    one.wait_stream(torch.cuda.current_stream())
    for c, b in zip(cs, bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=one):
            step(c, b)
        graphs.append(g)
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    _status_ok()
    for b, r in zip(bufs, eager):
        for k in b:
            assert torch.equal(b[k], r[k]), ("two graphs at once", k)
    c, b = cs[0], bufs[0]
    check_forward(c, b["GU"], b["Y"], b["O"])
    check_backward_input(c, b["GU"], b["dZ"], b["dGU"], b["dX"])
    check_weights(c, b["dZ"], b["Y"], b["dGU"], (b["dA"], b["da"], b["dB"], b["db"]))
    # new inputs under the same graph
    fresh = Case(T, c.h, c.ffn, "silu", 0.1, True, seed=9)
    for k in ("X", "A", "B", "a", "b", "dO"):
        getattr(c, k).copy_(getattr(fresh, k))
    graphs[0].replay()
    _status_ok()
    check_forward(c, b["GU"], b["Y"], b["O"])
    check_backward_input(c, b["GU"], b["dZ"], b["dGU"], b["dX"])


@pytest.mark.parametrize("T,h,ffn", [(3, 264, 520), (300, 2056, 2056), (1300, 2568, 1288)])
def test_without_dependent_launches_the_same_bits(T, h, ffn):
    """With each launch waiting for the one before to end (mlp_set_dependent_launch(0)): no bit changes, so no
    launch reads early what another still writes."""
    c = Case(T, h, ffn, "silu", 0.1, True)
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def step():
        GU, Y, O = torch.empty(T, 2 * ffn, **bf), torch.empty(T, ffn, **bf), torch.empty(T, h, **bf)
        dZ, dGU, dX = torch.empty(T, h, **bf), torch.empty(T, 2 * ffn, **bf), torch.empty(T, h, **bf)
        g = [torch.empty(s, device="cuda") for s in ((h, 2 * ffn), (2 * ffn,), (ffn, h), (h,))]
        for _ in range(3):
            c.fwd(GU, Y, O)
            c.bwd_input(GU, dZ, dGU, dX)
            c.bwd_weights(dZ, Y, dGU, *g)
        _status_ok()
        return [GU, Y, O, dZ, dGU, dX, *g]

    first = step()
    try:
        mlp.mlp_set_dependent_launch(False)
        second = step()
    finally:
        mlp.mlp_set_dependent_launch(True)
    for k, (a, b) in enumerate(zip(first, second)):
        assert torch.equal(a, b), k


# more elements than dropout's backward has threads (152 SMs * 16 CTAs * 128 threads * 8), so that its
# threads step on: over rows, over parts of rows, over rows of a single step
@pytest.mark.parametrize("T,h", [(3001, 1032), (1500, 5208), (330001, 8)])
def test_dropout_backward_of_many_elements(T, h):
    c = Case(T, h, 8)
    assert T * h > 152 * 16 * 128 * 8
    GU = torch.randn(T, 16, device="cuda").to(torch.bfloat16)
    (dZ, behind), dGU, dX = _guarded(T, h), torch.empty_like(GU), torch.empty_like(c.X)
    c.bwd_input(GU, dZ, dGU, dX)
    _status_ok()
    ref = f64(c.dO) * mlp_oracle.dropout_keep(T, h, c.p, SEED, OFFSET) * mlp_oracle.dropout_scale(c.p)
    # the scale and the product are each rounded to fp32 (2^-24), the result to bf16 (2^-8 of it)
    assert np.all(np.abs(f64(dZ) - ref) <= np.abs(ref) * (BF + 2.0**-22))
    assert torch.all(behind == 7)


def test_weights_written_just_before_the_call():
    """Weights that the launch right before the call writes (an optimizer step on the stream) are the ones used."""
    T, h, ffn = 5, 1032, 2744
    c = Case(T, h, ffn, "silu", 0.0, False)
    other = Case(T, h, ffn, "silu", 0.0, False, seed=8)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    outs = []
    for rounds in (1, 30):
        Y, O = torch.empty(T, ffn, **bf), torch.empty(T, h, **bf)
        for k in range(rounds):
            src = other if k % 2 else c
            c.X.copy_(c.X)
            A, B = (src.A, src.B)
            master = [x.float() for x in (A, B)]
            m, v = [torch.zeros_like(x) for x in master], [torch.ones_like(x) for x in master]
            wA, wB = torch.empty_like(A), torch.empty_like(B)
            for w, g, mm, vv in ((wA, master[0], m[0], v[0]), (wB, master[1], m[1], v[1])):
                mlp.adam_step(torch.zeros_like(g), g, mm, vv, w, lr=0.0)    # writes w = bf16(master)
            mlp.glu_fwd(h, ffn, 1, T, 0.0, SEED, OFFSET, ACT["silu"], c.X, wA, None, wB, None, None, None, Y, O)
            _status_ok()
            outs.append((k % 2, Y.clone(), O.clone()))
    for odd in (0, 1):
        same = [(y, o) for k, y, o in outs if k == odd]
        assert all(torch.equal(y, same[0][0]) and torch.equal(o, same[0][1]) for y, o in same)
    check_forward(c, None, outs[0][1], outs[0][2])


def test_threads_calling_at_once():
    """Two host threads, a stream each, the kernels' one-time set-up among their calls' work: the bits of one thread."""
    import threading
    cs = [Case(40, 520, 1096, "gelu", 0.1, True, seed=s) for s in (1, 2)]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    outs = [[torch.empty(40, n, **bf) for n in (2 * 1096, 1096, 520)] for _ in range(4)]
    for c, o in zip(cs, outs):
        c.fwd(*o)
    torch.cuda.synchronize()
    errors = []

    def work(c, o):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(50):
                    c.fwd(*o)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cs, outs[2:])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _status_ok()
    assert not errors
    for a, b in zip(outs[:2], outs[2:]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


FRESH = """
import sys
sys.path.insert(0, "tests")
import torch
import test_gpu_glu as t, test_gpu_qk_rope as q
from transformer_lm_megatron_gb300 import mlp
mlp.load()
for T in (3, 700):
    c, r = t.Case(T, 1032, 1544, "silu", 0.1, True), q.Case(T, 4, 2, 128)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    GU, Y, O = torch.empty(T, 2 * 1544, **bf), torch.empty(T, 1544, **bf), torch.empty(T, 1032, **bf)
    dZ, dGU, dX = torch.empty(T, 1032, **bf), torch.empty(T, 2 * 1544, **bf), torch.empty(T, 1032, **bf)
    (Qo, _), (Ko, _), (dQ, _), (dK, _) = r.out(4), r.out(2), r.out(4), r.out(2)
    w = r.grads()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.fwd(GU, Y, O)
        c.bwd_input(GU, dZ, dGU, dX)
        r.fwd(Qo, Ko)
        r.bwd(dQ, dK, w)
    g.replay()
    t._status_ok()
    t.check_forward(c, GU, Y, O)
    t.check_backward_input(c, GU, dZ, dGU, dX)
    q.check_fwd(r, Qo, Ko)
    q.check_bwd(r, dQ, dK, w)
print("captured first calls agree")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """A fresh process whose first calls are captured into a graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "agree" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_transposed_copies_change_no_bit():
    """scratch with mlp_set_wgrad_transpose(1): the weight gradients read transposed copies."""
    c = Case(1024, 1032, 1544, "silu")
    T, bf = c.T, dict(dtype=torch.bfloat16, device="cuda")
    Y = torch.randn(T, c.ffn, device="cuda").to(torch.bfloat16)
    dGU = torch.randn(T, 2 * c.ffn, device="cuda").to(torch.bfloat16)
    res = []
    try:
        for mode in (0, 1):
            mlp.mlp_set_wgrad_transpose(mode)
            dA, dB = torch.empty(c.h, 2 * c.ffn, device="cuda"), torch.empty(c.ffn, c.h, device="cuda")
            tr = mlp.Trace(capacity=16)
            tr.start()
            c.bwd_weights(c.dO, Y, dGU, dA, None, dB, None, scratch=torch.empty(T, c.h, device="cuda"))
            torch.cuda.synchronize()
            assert sum(k == 15 for k, _, _ in tr.stop()) == mode
            res.append((dA, dB))
    finally:
        mlp.mlp_set_wgrad_transpose(-1)
    _status_ok()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    check_weights(c, c.dO, Y, dGU, (res[0][0], None, res[0][1], None))


def test_gradient_against_differences():
    """The loss sum(O * dO) of the GPU's forward moves along a direction in X and the weights as the
    GPU's gradients say.  The step is 2^-3 of the weights' size, so that bf16's half steps (2^-8 each of
    O's values, about T h of them at random) stay under a tenth of the difference."""
    T, h, ffn = 64, 264, 328
    c = Case(T, h, ffn, "silu", 0.0, False, seed=4)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    GU, Y, O = torch.empty(T, 2 * ffn, **bf), torch.empty(T, ffn, **bf), torch.empty(T, h, **bf)
    dGU, dX = torch.empty(T, 2 * ffn, **bf), torch.empty(T, h, **bf)
    dA, dB = torch.empty(h, 2 * ffn, device="cuda"), torch.empty(ffn, h, device="cuda")
    c.fwd(GU, Y, O)
    c.bwd_input(GU, None, dGU, dX)
    c.bwd_weights(c.dO, Y, dGU, dA, None, dB, None)
    _status_ok()
    grads = {"X": dX.double(), "A": dA.double(), "B": dB.double()}
    base = {k: getattr(c, k).clone() for k in grads}
    for k, g in grads.items():
        # along the gradient itself: the difference is the largest there
        v = g / g.norm() * base[k].double().norm() * 2.0**-5
        lo, hi = (base[k].double() - v).to(torch.bfloat16), (base[k].double() + v).to(torch.bfloat16)
        loss = []
        for x in (lo, hi):
            getattr(c, k).copy_(x)
            c.fwd(GU, Y, O)
            torch.cuda.synchronize()
            loss.append((O.double() * c.dO.double()).sum().item())
        getattr(c, k).copy_(base[k])
        want = (g * (hi.double() - lo.double())).sum().item()
        # roundings of O: 2 T h values, each off by up to 2^-8 of it times dO (of size one), as a random sum
        noise = 4 * 2.0**-8 * np.sqrt(2 * T * h) * float(O.double().square().mean().sqrt())
        assert abs(loss[1] - loss[0] - want) <= noise + 0.05 * abs(want), (k, loss[1] - loss[0], want, noise)
    _status_ok()
