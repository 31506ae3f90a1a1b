"""GPU parity of the head norms with position rotation against the float64 oracle.

Bounds: sums of d squares in fp32 and the reciprocal root leave a normed value off by
2^-20 relative (d 2^-24 at most 2^-16 for the sum of positive terms, halved by the root
and far less with the sum as a tree; the bound takes 2^-17); a turned value combines two of
them with a sine and cosine off by 2^-22 (the angle is reduced exactly); so an output is off
by 2^-16 of the two elements' magnitudes, and by half a bf16 step, 2^-8 of itself.
dw: n = tokens * heads terms summed in fp32 as a tree: n 2^-24 of the terms' magnitudes at
the very most, and 2^-16 of each term from the above.
"""
import numpy as np
import pytest
import torch

from oracle import qk_rope_oracle as qro
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from gpu_harness import to_f64

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


def _status_ok():
    torch.cuda.synchronize()
    assert mlp.mlp_sync_status() == mlp.MLP_OK, mlp.last_error()


class Case:
    def __init__(self, T, nq, nk, d, rot=None, inter=False, sections=None, norm=True, far=0, gap=0, seed=0):
        """gap: elements between the heads of one token and the next token's, beyond the heads."""
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.T, self.nq, self.nk, self.d = T, nq, nk, d
        self.rot = d if rot is None else rot
        self.sections = [self.rot // 2] if sections is None else sections
        self.inter, self.norm, self.gap = inter, norm, gap
        self.Q, self.K, self.dQo, self.dKo = (self.view(r(T, n * d + gap), n) for n in (nq, nk, nq, nk))
        self.pos = (torch.randint(0, 5000, (len(self.sections), T), generator=g, dtype=torch.int32) + far).cuda()
        self.inv = (10000.0 ** -torch.linspace(0, 1, self.rot // 2, dtype=torch.float64)).float().cuda()
        self.wq, self.wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)) if norm else (None, None)
        self.kw = dict(wq=self.wq, wk=self.wk, eps=EPS, rot=self.rot, sections=self.sections, interleaved=inter)

    def view(self, flat, n):
        return flat[:, : n * self.d].view(self.T, n, self.d)

    def out(self, n):
        """A [T, n, d] view with the case's gap, NaN inside, 7 in the gaps and behind: (view, whole)."""
        whole = torch.full((self.T + 3, n * self.d + self.gap), 7.0, dtype=torch.bfloat16, device="cuda")
        v = self.view(whole[: self.T], n)
        v.fill_(float("nan"))
        return v, whole

    def untouched(self, whole, n):
        w = whole.clone()
        w[: self.T, : n * self.d] = 7
        return bool(torch.all(w == 7))

    def fwd(self, Qo, Ko, Q=None, K=None, stream=None):
        mlp.qk_norm_rope_fwd(self.Q if Q is None else Q, self.K if K is None else K, Qo, Ko, self.pos, self.inv, stream=stream, **self.kw)

    def grads(self):
        if not self.norm:
            return dict(dwq=None, dwk=None, ws=None)
        nan = lambda n: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
        return dict(dwq=nan(self.d), dwk=nan(self.d), ws=nan(mlp.qk_norm_rope_workspace(self.d)))

    def bwd(self, dQ, dK, w, accumulate=False, dQo=None, dKo=None, stream=None):
        q, k = (self.Q, self.K) if self.norm else (None, None)
        mlp.qk_norm_rope_bwd(q, k, self.dQo if dQo is None else dQo, self.dKo if dKo is None else dKo, dQ, dK, self.pos, self.inv,
                             accumulate=accumulate, stream=stream, **w, **self.kw)

    def angles(self):
        return qro.angles(self.pos.cpu().numpy(), self.inv.cpu().numpy(), self.sections)

    def partner(self, m):
        """Each element's magnitude plus its pair's."""
        i, j = (np.arange(0, self.rot, 2), np.arange(1, self.rot, 2)) if self.inter else (np.arange(self.rot // 2), np.arange(self.rot // 2) + self.rot // 2)
        s = m.copy()
        s[..., i] = s[..., j] = m[..., i] + m[..., j]
        return s


def _near(got, ref, bound, what):
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - ref) - bound
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, (what, at, got[at], ref[at], bound[at])


def check_fwd(c, Qo, Ko, Q=None, K=None):
    ang = c.angles()
    for got, x, w, what in ((Qo, c.Q if Q is None else Q, c.wq, "Qo"), (Ko, c.K if K is None else K, c.wk, "Ko")):
        x, w = to_f64(x), None if w is None else to_f64(w)
        n = x if w is None else x * qro.rstd(x, EPS) * w
        ref = qro.turn(n, ang, c.rot, c.inter)
        _near(to_f64(got), ref, 2.0**-8 * np.abs(ref) + 2.0**-15 * c.partner(np.abs(n)), what)


def check_bwd(c, dQ, dK, w, before=None):
    ang = c.angles()
    for got, x, wt, dy, dw, what in ((dQ, c.Q, c.wq, c.dQo, w["dwq"], "q"), (dK, c.K, c.wk, c.dKo, w["dwk"], "k")):
        x, dy, wt = to_f64(x), to_f64(dy), None if wt is None else to_f64(wt)
        ref, ref_w = qro.bwd(x, wt, dy, ang, c.rot, c.inter, EPS)
        size = c.partner(np.abs(dy))
        if wt is not None:
            r = qro.rstd(x, EPS)
            g = size  # at least the turned gradient's magnitude
            wg = np.abs(wt) * g
            size = r * wg + np.abs(x) * r**3 * (wg * np.abs(x)).mean(-1, keepdims=True)
            n = c.T * x.shape[1]
            old = 0.0 if before is None else to_f64(before["dw" + what])
            bound = (n * 2.0**-24 + 2.0**-15) * (g * np.abs(x) * r).sum((0, 1)) + 2.0**-22 * (np.abs(ref_w) + np.abs(old))
            _near(to_f64(dw), ref_w + old, bound, "dw" + what)
        _near(to_f64(got), ref, 2.0**-8 * np.abs(ref) + 2.0**-15 * size, "d" + what)


FORMS = [
    # T, nq, nk, d, rot, interleaved, sections, norm, far, gap
    (1, 1, 1, 8, 8, False, None, True, 0, 0),
    (1, 32, 8, 128, 128, False, None, True, 1000000, 0),
    (3, 4, 4, 64, 64, True, [16, 8, 8], True, 0, 64),
    (7, 5, 1, 80, 80, False, [20, 20], True, 4000000, 8),
    (13, 3, 2, 72, 72, True, None, True, 0, 0),
    (70, 8, 2, 96, 48, False, [8, 8, 8], True, 0, 96),
    (33, 6, 3, 160, 160, False, None, True, -2500, 160),
    (19, 2, 2, 192, 128, True, [1, 62, 1], True, 0, 0),
    (11, 3, 1, 256, 256, False, [128, 0, 0], True, 0, 0),
    (9, 7, 7, 248, 8, False, None, True, 0, 0),
    (40, 9, 2, 24, 16, True, [0, 8], True, 0, 8),
    (501, 16, 4, 128, 128, False, [16, 24, 24], True, 0, 512),
    (1500, 33, 3, 64, 64, False, None, True, 120000, 0),
    (5, 4, 2, 80, 48, True, [12, 12], False, 0, 0),
    (130, 5, 5, 128, 64, False, [10, 11, 11], False, 2000000, 128),
    (2, 2, 1, 40, 40, False, None, False, 0, 0),
]


@pytest.mark.parametrize("T,nq,nk,d,rot,inter,sections,norm,far,gap", FORMS)
def test_forward_and_backward(T, nq, nk, d, rot, inter, sections, norm, far, gap):
    c = Case(T, nq, nk, d, rot, inter, sections, norm, far, gap)
    (Qo, wq), (Ko, wk) = c.out(nq), c.out(nk)
    c.fwd(Qo, Ko)
    _status_ok()
    check_fwd(c, Qo, Ko)
    assert c.untouched(wq, nq) and c.untouched(wk, nk)
    (dQ, wq), (dK, wk) = c.out(nq), c.out(nk)
    w = c.grads()
    c.bwd(dQ, dK, w)
    _status_ok()
    check_bwd(c, dQ, dK, w)
    assert c.untouched(wq, nq) and c.untouched(wk, nk)
    if norm:
        before = dict(dwq=torch.randn(d, device="cuda"), dwk=torch.randn(d, device="cuda"))
        w2 = dict(dwq=before["dwq"].clone(), dwk=before["dwk"].clone(), ws=w["ws"])
        c.bwd(dQ, dK, w2, accumulate=True)
        _status_ok()
        check_bwd(c, dQ, dK, w2, before)


@pytest.mark.parametrize("norm", [True, False])
def test_in_place(norm):
    c = Case(37, 6, 2, 128, norm=norm, gap=64)
    (Qo, _), (Ko, _) = c.out(6), c.out(2)
    c.fwd(Qo, Ko)
    q, k = c.Q.clone(), c.K.clone()
    mlp.qk_norm_rope_fwd(q, k, q, k, c.pos, c.inv, **c.kw)
    (dQ, _), (dK, _) = c.out(6), c.out(2)
    w, w2 = c.grads(), c.grads()
    c.bwd(dQ, dK, w)
    g, h = c.dQo.clone(), c.dKo.clone()
    c.bwd(g, h, w2, dQo=g, dKo=h)
    _status_ok()
    assert torch.equal(q, Qo) and torch.equal(k, Ko) and torch.equal(g, dQ) and torch.equal(h, dK)
    if norm:
        assert torch.equal(w["dwq"], w2["dwq"]) and torch.equal(w["dwk"], w2["dwk"])


def test_positions_at_the_ends_of_their_type():
    """Any int32 position: the angle is the exact product modulo a turn, off by the frequency's 2^-64 of a
    turn times the position and by the 2^-32 of a turn that its top 32 bits leave out."""
    c = Case(6, 2, 2, 64, norm=False)
    c.pos = torch.tensor([[0, 2**31 - 1, -2**31, 2**24 + 1, -1, 123456789]], dtype=torch.int32, device="cuda")
    (Qo, _), (Ko, _) = c.out(2), c.out(2)
    c.fwd(Qo, Ko)
    _status_ok()
    check_fwd(c, Qo, Ko)


def test_heads_of_zeros_and_of_nan():
    """A head of zeros stays zeros (eps keeps the norm finite), its gradient is finite; a NaN reaches its own head only."""
    c = Case(5, 6, 2, 96)
    c.Q[1, 2] = 0
    c.Q[3, 4, 17] = float("nan")
    (Qo, _), (Ko, _) = c.out(6), c.out(2)
    c.fwd(Qo, Ko)
    (dQ, _), (dK, _) = c.out(6), c.out(2)
    w = c.grads()
    c.bwd(dQ, dK, w)
    _status_ok()
    assert torch.all(Qo[1, 2] == 0)
    bad = torch.isnan(Qo).any(-1)
    assert bad.sum() == 1 and bool(bad[3, 4]) and not torch.isnan(Ko).any()
    bad = torch.isnan(dQ).any(-1)
    assert bad.sum() == 1 and bool(bad[3, 4]) and not torch.isnan(dK).any()
    assert torch.isnan(w["dwq"]).any() and not torch.isnan(w["dwk"]).any()


def test_many_rows_take_the_large_offsets():
    """A row stride that puts the last token's offset beyond 2^31 elements."""
    T, ld = 9, 1 << 28
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    c = Case(T, 2, 1, 64)
    Qo = big[:, : 2 * 64].view(T, 2, 64)
    Ko = big[:, 4096 : 4096 + 64].view(T, 1, 64)
    Qo.fill_(float("nan"))
    Ko.fill_(float("nan"))
    c.fwd(Qo, Ko)
    _status_ok()
    check_fwd(c, Qo, Ko)
    (dQ, _), (dK, _) = c.out(2), c.out(1)
    w = c.grads()
    g, h = Qo.clone(), Ko.clone()
    c.dQo, c.dKo = g, h
    c.bwd(dQ, dK, w, dQo=Qo, dKo=Ko)
    _status_ok()
    check_bwd(c, dQ, dK, w)


@pytest.mark.parametrize("T", [1, 300])
def test_graphs_streams_and_repeats_give_the_same_bits(T):
    cs = [Case(T, 8, 2, 128, seed=s, gap=128) for s in (1, 2)]

    def buffers(c):
        return dict(Qo=c.out(8)[0], Ko=c.out(2)[0], dQ=c.out(8)[0], dK=c.out(2)[0], **c.grads())

    def step(c, b):
        c.fwd(b["Qo"], b["Ko"])
        c.bwd(b["dQ"], b["dK"], {k: b[k] for k in ("dwq", "dwk", "ws")})

    ref = [buffers(c) for c in cs]
    for c, b in zip(cs, ref):
        step(c, b)
    _status_ok()
    streams, again = [torch.cuda.Stream() for _ in cs], [buffers(c) for c in cs]
    torch.cuda.synchronize()
    for s, c, b in zip(streams, cs, again):
        with torch.cuda.stream(s):
            for _ in range(3):
                step(c, b)
    graphs, bufs = [], [buffers(c) for c in cs]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    for c, b in zip(cs, bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=one):
            step(c, b)
        graphs.append(g)
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    _status_ok()
    for other in (again, bufs):
        for b, r in zip(other, ref):
            for k in b:
                if k != "ws":
                    assert torch.equal(b[k], r[k]), k


def test_gradient_against_differences():
    """sum(y * dy) of the GPU's forward along the gradient, where the rounding of y's T n d values to
    bf16 (2^-8 each at most, at random) is under the bound and the curvature within a twentieth."""
    c = Case(40, 4, 4, 64, seed=6)
    (Qo, _), (Ko, _), (dQ, _), (dK, _) = c.out(4), c.out(4), c.out(4), c.out(4)
    w = c.grads()
    c.bwd(dQ, dK, w)
    _status_ok()
    for x, g in ((c.Q, dQ.double()), (c.wk, w["dwk"].double())):
        base = x.clone()
        v = g / g.norm() * base.double().norm() * 2.0**-5
        lo, hi = (base.double() - v).to(torch.bfloat16), (base.double() + v).to(torch.bfloat16)
        loss = []
        for y in (lo, hi):
            x.copy_(y)
            c.fwd(Qo, Ko)
            torch.cuda.synchronize()
            loss.append(((Qo.double() * c.dQo.double()).sum() + (Ko.double() * c.dKo.double()).sum()).item())
        x.copy_(base)
        want = (g * (hi.double() - lo.double())).sum().item()
        noise = 4 * 2.0**-8 * np.sqrt(2 * 2 * c.T * 4 * 64)
        assert abs(loss[1] - loss[0] - want) <= noise + 0.05 * abs(want), (loss, want, noise)
