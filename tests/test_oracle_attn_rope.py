"""Pins of the oracle of the attention block with head norms and rotation."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ato
from oracle import attn_rope_oracle as aro
from oracle import qk_rope_oracle as qro


def _case(T=12, h=32, nh=2, seed=2):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)  # noqa: E731
    return r(T, h), 0.3 * r(h, 3 * h), 0.3 * r(3 * h), 0.3 * r(h, h), 0.3 * r(h), r(T, h), r(16), r(16)


def test_no_norm_and_no_angle_is_the_plain_block():
    X, Wqkv, bqkv, Wo, bo, dOut, _, _ = _case()
    rope = dict(wq=None, wk=None, ang=np.zeros((12, 8)), rot=16, inter=False, eps=0.0)
    a = ato.attn_fwd(X, Wqkv, bqkv, Wo, bo, 2, 1, 6, 0.1, 7, token_offset=3)
    b = aro.fwd(X, Wqkv, bqkv, Wo, bo, 2, 6, 0.1, 7, rope, token_offset=3)
    for k in ("QKV", "P", "O", "out"):
        np.testing.assert_allclose(b[k], a[k], rtol=1e-12, atol=1e-12)
    x = ato.attn_bwd(dOut, X, Wqkv, Wo, a["QKV"], a["P"], a["O"], a["keep"], 2, 1, 6, 0.1)
    y = aro.bwd(dOut, X, Wqkv, Wo, b, 2, 6, 0.1, rope)
    for k in ("dQKV", "dX", "dWqkv", "dbqkv", "dWo", "dbo"):
        np.testing.assert_allclose(y[k], x[k], rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("inter", [False, True])
def test_against_autograd(inter):
    X, Wqkv, bqkv, Wo, bo, dOut, wq, wk = _case()
    T, h, nh, L, d, rot = 12, 32, 2, 6, 16, 8
    ang = qro.angles(np.random.default_rng(0).integers(0, 99, (2, T)), np.linspace(0.1, 1, 4).astype(np.float32), [1, 3])
    rope = dict(wq=wq, wk=wk, ang=ang, rot=rot, inter=inter, eps=1e-5)
    fw = aro.fwd(X, Wqkv, bqkv, Wo, bo, nh, L, 0.1, 7, rope)
    bw = aro.bwd(dOut, X, Wqkv, Wo, fw, nh, L, 0.1, rope)
    leaf = {k: torch.tensor(v, requires_grad=True) for k, v in dict(X=X, Wqkv=Wqkv, bqkv=bqkv, Wo=Wo, bo=bo, wq=wq, wk=wk).items()}
    c, s = torch.tensor(np.cos(ang))[:, None], torch.tensor(np.sin(ang))[:, None]

    def turned(x, w):
        x = x.view(T, nh, d)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        y = x.clone()
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
        return y

    QKV = leaf["X"] @ leaf["Wqkv"] + leaf["bqkv"]
    q, k, v = turned(QKV[:, :h], leaf["wq"]), turned(QKV[:, h:2 * h], leaf["wk"]), QKV[:, 2 * h:].view(T, nh, d)
    q, k, v = (x.view(T // L, L, nh, d).transpose(1, 2) for x in (q, k, v))
    O = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True).transpose(1, 2).reshape(T, h)
    out = leaf["X"] + torch.where(torch.tensor(fw["keep"]), (O @ leaf["Wo"] + leaf["bo"]) / (1 - float(np.float32(0.1))), 0.0)
    np.testing.assert_allclose(fw["out"], out.detach().numpy(), rtol=1e-6, atol=1e-6)
    out.backward(torch.tensor(dOut))
    for k in ("X", "Wqkv", "bqkv", "Wo", "bo", "wq", "wk"):
        np.testing.assert_allclose(bw["d" + k], leaf[k].grad.numpy(), rtol=1e-6, atol=1e-6, err_msg=k)
