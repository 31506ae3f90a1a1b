"""The attention block with head norms and rotation, and a decoder layer of it and the
gated feed-forward block, on the GPU against the float64 oracles.

Bars as in test_gpu_attn: bf16 tensors within 1e-2 of the bf16-mirroring oracle
(max|gpu - oracle| / max|oracle|), fp32 gradients within the oracle's own distance
between its mirroring and exact modes (never below 1e-3), and that distance more from
the exact mode.  The norm weights' gradients sum products of the core's bf16 gradients,
like dbqkv, and are held to the fp32 bar.
"""
import numpy as np
import pytest
import torch

from oracle import attn_rope_oracle as aro
from oracle import glu_oracle as glo
from oracle import qk_rope_oracle as qro
from oracle.mlp_oracle import round_bf16
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from gpu_harness import BF16_TOL, F32_TOL, bits_f64, rel_err, to_f64

pytestmark = pytest.mark.gpu

P, SEED = 0.1, 1234


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


@pytest.fixture
def attn_core(request):
    mlp.mlp_set_attn_fused(request.param == "fused")
    yield request.param
    mlp.mlp_set_attn_fused(True)


def _randn(g, *s, k=1.0):
    return (torch.randn(*s, generator=g) * k).to(torch.bfloat16)


class Layer:
    """An attention block's weights, its rotation and buffers."""

    def __init__(self, T, h, nh, L, rot, inter, sections, norm, seed=3):
        g = torch.Generator().manual_seed(seed)
        self.T, self.h, self.nh, self.L, self.d = T, h, nh, L, h // nh
        k = 0.5 / np.sqrt(h)
        self.w = (_randn(g, h, 3 * h, k=k), _randn(g, 3 * h, k=k), _randn(g, h, h, k=k), _randn(g, h, k=k))
        self.wq, self.wk = ((1 + 0.2 * torch.randn(self.d, generator=g)).to(torch.bfloat16) for _ in range(2)) if norm else (None, None)
        self.pos = torch.arange(T, dtype=torch.int32).remainder(L)[None].repeat(len(sections), 1) + torch.randint(
            0, 300, (len(sections), 1), generator=g, dtype=torch.int32)
        self.inv = (10000.0 ** -torch.linspace(0, 1, rot // 2, dtype=torch.float64)).float()
        cu = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.dev = tuple(x.cuda() for x in self.w)
        self.rope = mlp.Rope(self.d, self.pos.cuda(), self.inv.cuda(), cu(self.wq), cu(self.wk), rot=rot, sections=sections,
                             interleaved=inter)
        self.buf = mlp.AttnBuffers(T, h, nh, L)
        self.QKr = torch.empty(T, 2 * h, dtype=torch.bfloat16, device="cuda")
        self.oracle = dict(wq=None if not norm else bits_f64(self.wq), wk=None if not norm else bits_f64(self.wk),
                           ang=qro.angles(self.pos.numpy(), self.inv.numpy(), sections), rot=rot, inter=inter, eps=1e-6)

    def fwd(self, X, off=0):
        b = self.buf
        mlp.attn_rope_fwd(self.h, self.nh, 1, self.T, self.L, P, SEED, off, self.rope, X, *self.dev, None, b.QKV, self.QKr, b.S, b.P,
                          b.O, b.out)
        return b.out

    def bwd(self, X, dOut, accumulate=False, off=0):
        b = self.buf
        mlp.attn_rope_bwd(self.h, self.nh, 1, self.T, self.L, P, SEED, off, self.rope, 1, accumulate, dOut, X, self.dev[0], self.dev[2],
                          b.QKV, self.QKr, b.P, b.O, b.dZ, b.dO, b.dP, b.dS, b.dQKV, b.dX, b.dWqkv, b.dbqkv, b.dWo, b.dbo)
        return b.dX

    def ref(self, X, dOut, mirror, off=0):
        w = [bits_f64(x) for x in self.w]
        fw = aro.fwd(X, *w, self.nh, self.L, P, SEED, self.oracle, token_offset=off, mirror=mirror)
        return fw, aro.bwd(dOut, X, w[0], w[2], fw, self.nh, self.L, P, self.oracle, mirror=mirror)

    def grads(self):
        b = self.buf
        got = {k: to_f64(getattr(b, k)) for k in ("dWqkv", "dbqkv", "dWo", "dbo")}
        if self.wq is not None:
            got.update(dwq=to_f64(self.rope.dwq), dwk=to_f64(self.rope.dwk))
        return got


def _status_ok():
    torch.cuda.synchronize()
    assert mlp.mlp_sync_status() == mlp.MLP_OK, mlp.last_error()


def _compare(got, mirror, pure, bar, what):
    e, gap = rel_err(got, mirror), rel_err(mirror, pure)
    if bar is None:
        bar = max(F32_TOL, gap)
    assert e <= bar, (what, "mirror", e, bar)
    e = rel_err(got, pure)
    assert e <= bar + gap, (what, "exact", e, bar + gap)


@pytest.mark.parametrize("attn_core", ["fused", "unfused"], indirect=True)
@pytest.mark.parametrize("T,h,nh,L,rot,inter,sections,norm,k", [
    (256, 256, 4, 128, 64, False, [32], True, 2),          # two micro-batches accumulated
    (272, 320, 4, 136, 48, True, [8, 8, 8], True, 1),      # d = 80, three axes, part of the head turned
    (8, 128, 2, 8, 64, False, [32], True, 1),
    (384, 640, 8, 384, 80, False, [20, 20], False, 1),     # the rotation alone
    (200, 432, 2, 200, 216, False, [108], True, 1),        # d = 216: above the fused core's head size
])
def test_attention_block(T, h, nh, L, rot, inter, sections, norm, k, attn_core):
    y = Layer(T, h, nh, L, rot, inter, sections, norm)
    g = torch.Generator().manual_seed(8)
    acc = {}
    for j in range(k):
        X, dOut = _randn(g, T, h), _randn(g, T, h)
        y.fwd(X.cuda(), j * T)
        y.bwd(X.cuda(), dOut.cuda(), accumulate=j > 0, off=j * T)
        _status_ok()
        (fm, bm), (fp, bp) = (y.ref(bits_f64(X), bits_f64(dOut), m, j * T) for m in (True, False))
        for name in ("QKV", "P", "O", "out"):
            _compare(to_f64(getattr(y.buf, name)), fm[name], fp[name], BF16_TOL, name)
        _compare(to_f64(y.QKr), fm["QKr"], fp["QKr"], BF16_TOL, "QKr")
        for name in ("dQKV", "dX"):
            _compare(to_f64(getattr(y.buf, name)), bm[name], bp[name], BF16_TOL, name)
        for n in y.grads():
            m, p = acc.get(n, (0.0, 0.0))
            acc[n] = (m + bm[n], p + bp[n])
    for n, got in y.grads().items():
        _compare(got, *acc[n], None, n)


def test_without_norm_and_angle_equals_the_plain_block():
    """All frequencies zero and no norm: the turned queries and keys are the projection's, and every
    output has attn_step's bits."""
    T, h, nh, L = 256, 256, 4, 128
    y = Layer(T, h, nh, L, 64, False, [32], False)
    y.rope.inv_freq.zero_()
    g = torch.Generator().manual_seed(8)
    X, dOut = _randn(g, T, h).cuda(), _randn(g, T, h).cuda()
    y.fwd(X)
    y.bwd(X, dOut)
    plain = mlp.AttnBuffers(T, h, nh, L)
    mlp.attn_step(h, nh, 1, L, P, SEED, y.dev, X, dOut, plain, accumulate=False)
    _status_ok()
    assert torch.equal(y.QKr, plain.QKV[:, :2 * h])
    for n in ("QKV", "P", "O", "out", "dQKV", "dX", "dWqkv", "dbqkv", "dWo", "dbo"):
        assert torch.equal(getattr(y.buf, n), getattr(plain, n)), n


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_decoder_layer(act):
    """X -> attention block with norms and rotation -> gated block, and back: every gradient of
    both blocks from the gradient of the layer's output, against the chain of the oracles."""
    T, h, nh, L, ffn = 272, 320, 4, 136, 872
    y = Layer(T, h, nh, L, 80, False, [16, 12, 12], True)
    g = torch.Generator().manual_seed(11)
    k = 1 / np.sqrt(h)
    A, a, B, b = _randn(g, h, 2 * ffn, k=k), _randn(g, 2 * ffn, k=k), _randn(g, ffn, h, k=1 / np.sqrt(ffn)), _randn(g, h, k=k)
    X, dOut = _randn(g, T, h), _randn(g, T, h)
    bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
    GU, Y, O = torch.empty(T, 2 * ffn, **bf), torch.empty(T, ffn, **bf), torch.empty(T, h, **bf)
    dZ, dGU, dH = torch.empty(T, h, **bf), torch.empty(T, 2 * ffn, **bf), torch.empty(T, h, **bf)
    dA, da, dB, db = torch.empty(h, 2 * ffn, **f32), torch.empty(2 * ffn, **f32), torch.empty(ffn, h, **f32), torch.empty(h, **f32)
    code = mlp.GLU_SILU if act == "silu" else mlp.GLU_GELU
    Ad, ad, Bd, bd, Xd, dOd = (x.cuda() for x in (A, a, B, b, X, dOut))
    H = y.fwd(Xd)
    mlp.glu_fwd(h, ffn, 1, T, P, SEED + 1, 0, code, H, Ad, ad, Bd, bd, None, GU, Y, O)
    mlp.glu_bwd_input(h, ffn, 1, T, P, SEED + 1, 0, code, 1, dOd, Ad, Bd, GU, dZ, dGU, dH)
    y.bwd(Xd, dH)
    mlp.glu_bwd_weights(h, ffn, 1, T, 0, H, dZ, Y, dGU, dA, da, dB, db)
    _status_ok()
    A64, a64, B64, b64, X64, d64 = (bits_f64(x) for x in (A, a, B, b, X, dOut))
    W = [bits_f64(x) for x in y.w]
    ref = {}
    for mirror in (True, False):
        rb = round_bf16 if mirror else (lambda v: v)
        fw = aro.fwd(X64, *W, nh, L, P, SEED, y.oracle, mirror=mirror)
        h64 = fw["out"]
        gu32 = glo.gates(h64, A64, a64)
        gu, yy = rb(gu32), rb(glo.gated(gu32, act))
        o = rb(glo.out(yy, B64, b64, h64, P, SEED + 1))
        z = rb(glo.d_out(d64, P, SEED + 1))
        dgu = rb(glo.d_gates(z, B64, gu, act))
        dh = rb(glo.d_input(dgu, A64, d64))
        r = dict(zip(("dA", "da", "dB", "db"), glo.d_weights(h64, z, yy, dgu)))
        r.update(out=h64, O=o, dH=dh, **aro.bwd(dh, X64, W[0], W[2], fw, nh, L, P, y.oracle, mirror=mirror))
        ref[mirror] = r
    got = {**y.grads(), **{n: to_f64(v) for n, v in dict(dA=dA, da=da, dB=dB, db=db, out=H, O=O, dH=dH, dX=y.buf.dX).items()}}
    for n, v in got.items():
        _compare(v, ref[True][n], ref[False][n], BF16_TOL if n in ("out", "O", "dH", "dX") else None, n)
