"""Refusals of the gated block's, the head norms' and the rotating attention's entry
points, through the C ABI and the binding, before anything touches a device."""
import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

GOOD = 4096  # an aligned fake address: validation fails before anything reads it


@pytest.fixture(scope="module")
def lib():
    gb_build.build()
    return mlp.load()


GLU_FWD = dict(h=64, ffn=256, t=2, tokens=16, p=0.1, seed=1, off=0, act=0, X=GOOD, A=GOOD, a=GOOD, B=GOOD, b=GOOD, R=GOOD, GU=GOOD,
               Y=GOOD, O=GOOD, stream=None)
GLU_IN = dict(h=64, ffn=256, t=2, tokens=16, p=0.1, seed=1, off=0, act=0, res=1, dO=GOOD, A=GOOD, B=GOOD, GU=GOOD, dZ=GOOD, dGU=GOOD,
              dX=GOOD, stream=None)
GLU_W = dict(h=64, ffn=256, t=2, tokens=16, acc=1, X=GOOD, dZ=GOOD, Y=GOOD, dGU=GOOD, dA=GOOD, da=GOOD, dB=GOOD, db=GOOD, scratch=GOOD,
             stream=None)
ROPE = dict(rot=64, inter=0, axes=1, s0=32, s1=0, s2=0, eps=1e-6, wq=GOOD, wk=GOOD, pos=GOOD, inv=GOOD)
QK_FWD = dict(tokens=16, nq=4, nk=2, d=64, **ROPE, Q=GOOD, ldq=256, K=GOOD, ldk=128, Qo=GOOD, ldqo=256, Ko=GOOD, ldko=128, stream=None)
QK_BWD = dict(tokens=16, nq=4, nk=2, d=64, **ROPE, acc=1, Q=GOOD, ldq=256, K=GOOD, ldk=128, dQo=GOOD, lddqo=256, dKo=GOOD, lddko=128,
              dQ=GOOD, lddq=256, dK=GOOD, lddk=128, dwq=GOOD, dwk=GOOD, ws=GOOD, stream=None)
ATTN = dict(h=256, nh=4, t=2, tokens=64, seq=32, p=0.1, seed=1, off=0, **ROPE)
ATTN_FWD = dict(**ATTN, X=GOOD, Wqkv=GOOD, bqkv=GOOD, Wo=GOOD, bo=GOOD, R=None, QKV=GOOD, QKr=GOOD, S=GOOD, P=GOOD, O=GOOD, out=GOOD,
                stream=None)
ATTN_BWD = dict(**ATTN, res=1, acc=1, **{k: GOOD for k in ("dOut X Wqkv Wo QKV QKr P O dZ dO dP dS dQKV dX dWqkv dbqkv dWo dbo dwq dwk "
                                                           "ws").split()}, stream=None)
EINVAL, EALIGN, EUNS = mlp.MLP_EINVAL, mlp.MLP_EALIGN, mlp.MLP_EUNSUPPORTED

BAD_GLU = [(dict(h=0), EINVAL), (dict(h=12), EINVAL), (dict(ffn=0), EINVAL), (dict(ffn=252), EINVAL), (dict(t=0), EINVAL),
           (dict(t=3), EINVAL), (dict(t=64), EINVAL), (dict(tokens=0), EINVAL), (dict(tokens=-1), EINVAL), (dict(tokens=1 << 31), EINVAL), (dict(tokens=(1 << 30) + 1), EINVAL),
           (dict(ffn=(1 << 29) + 8, t=1), EINVAL)]
BAD_ACT = [(dict(act=2), EINVAL), (dict(act=-1), EINVAL), (dict(p=1.0), EINVAL), (dict(p=-0.5), EINVAL), (dict(p=float("nan")), EINVAL)]
BAD_ROPE = [(dict(rot=0), EINVAL), (dict(rot=60), EINVAL), (dict(rot=72, s0=36), EINVAL), (dict(inter=2), EINVAL), (dict(axes=0), EINVAL),
            (dict(axes=4), EINVAL), (dict(s0=31), EINVAL), (dict(s0=33, s1=-1), EINVAL), (dict(s0=16, s1=16), EINVAL),
            (dict(axes=2, s0=16, s1=8, s2=8), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(wq=None), EINVAL),
            (dict(wk=None), EINVAL), (dict(wq=GOOD + 8), EALIGN), (dict(pos=None), EINVAL), (dict(inv=None), EINVAL),
            (dict(pos=GOOD + 2), EALIGN), (dict(inv=GOOD + 1), EALIGN)]


def _refuse(lib, name, base, kw, code):
    args = {**base, **kw}
    assert set(args) == set(base)
    assert getattr(lib, name)(*args.values()) == code
    assert mlp.last_error()


@pytest.mark.parametrize("kw,code", BAD_GLU + BAD_ACT + [(dict(X=None), EINVAL), (dict(A=None), EINVAL), (dict(B=None), EINVAL),
                                                         (dict(Y=None), EINVAL), (dict(O=None), EINVAL), (dict(a=GOOD + 8), EALIGN),
                                                         (dict(b=GOOD + 2), EALIGN), (dict(R=GOOD + 8), EALIGN),
                                                         (dict(GU=GOOD + 8), EALIGN), (dict(X=GOOD + 4), EALIGN)])
def test_glu_fwd(lib, kw, code):
    _refuse(lib, "glu_fwd", GLU_FWD, kw, code)


@pytest.mark.parametrize("kw,code", BAD_GLU + BAD_ACT + [({k: None}, EINVAL) for k in ("dO", "A", "B", "GU", "dZ", "dGU", "dX")]
                         + [(dict(dZ=GOOD + 8), EALIGN), (dict(dGU=GOOD + 8), EALIGN)])
def test_glu_bwd_input(lib, kw, code):
    _refuse(lib, "glu_bwd_input", GLU_IN, kw, code)


@pytest.mark.parametrize("kw,code", BAD_GLU + [({k: None}, EINVAL) for k in ("X", "dZ", "Y", "dGU", "dA", "dB")]
                         + [({k: GOOD + 8}, EALIGN) for k in ("dA", "da", "db", "scratch")])
def test_glu_bwd_weights(lib, kw, code):
    _refuse(lib, "glu_bwd_weights", GLU_W, kw, code)


BAD_QK = BAD_ROPE + [(dict(tokens=0), EINVAL), (dict(tokens=1 << 31), EINVAL), (dict(nq=0), EINVAL), (dict(nk=0), EINVAL),
                     (dict(nk=-1), EINVAL), (dict(d=0), EINVAL), (dict(d=60, ldq=256), EINVAL),
                     (dict(d=264, rot=64), EUNS)]


@pytest.mark.parametrize("kw,code", BAD_QK + [({k: None}, EINVAL) for k in ("Q", "K", "Qo", "Ko")]
                         + [({k: GOOD + 8}, EALIGN) for k in ("Q", "K", "Qo", "Ko")]
                         + [({k: 120}, EINVAL) for k in ("ldq", "ldk", "ldqo", "ldko")] + [(dict(ldq=260), EINVAL)])
def test_qk_norm_rope_fwd(lib, kw, code):
    _refuse(lib, "qk_norm_rope_fwd", QK_FWD, kw, code)


@pytest.mark.parametrize("kw,code", BAD_QK + [({k: None}, EINVAL) for k in ("Q", "K", "dQo", "dKo", "dQ", "dK", "dwq", "dwk", "ws")]
                         + [({k: GOOD + 8}, EALIGN) for k in ("Q", "dQo", "dK", "ws")]
                         + [({k: 120}, EINVAL) for k in ("ldq", "ldk", "lddqo", "lddko", "lddq", "lddk")])
def test_qk_norm_rope_bwd(lib, kw, code):
    _refuse(lib, "qk_norm_rope_bwd", QK_BWD, kw, code)


BAD_ATTN = BAD_ROPE + [(dict(h=96, nh=16), EINVAL), (dict(tokens=60), EINVAL), (dict(t=3), EINVAL), (dict(p=1.0), EINVAL),
                       (dict(h=544, nh=2, t=1), EUNS), (dict(QKr=None), EINVAL), (dict(QKr=GOOD + 8), EALIGN), (dict(QKV=None), EINVAL)]


@pytest.mark.parametrize("kw,code", BAD_ATTN + [(dict(X=None), EINVAL), (dict(R=GOOD + 8), EALIGN)])
def test_attn_rope_fwd(lib, kw, code):
    _refuse(lib, "attn_rope_fwd", ATTN_FWD, kw, code)


@pytest.mark.parametrize("kw,code", BAD_ATTN + [(dict(dwq=None), EINVAL), (dict(ws=None), EINVAL), (dict(dX=None), EINVAL)])
def test_attn_rope_bwd(lib, kw, code):
    _refuse(lib, "attn_rope_bwd", ATTN_BWD, kw, code)


def test_valid_calls_without_a_gpu_report_unsupported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, base in (("glu_fwd", GLU_FWD), ("glu_bwd_input", GLU_IN), ("glu_bwd_weights", GLU_W), ("qk_norm_rope_fwd", QK_FWD),
                       ("qk_norm_rope_bwd", QK_BWD), ("attn_rope_fwd", ATTN_FWD), ("attn_rope_bwd", ATTN_BWD)):
        assert getattr(lib, name)(*base.values()) == EUNS, name
    none = dict(wq=None, wk=None, Q=None, K=None, ldq=0, ldk=0, dwq=None, dwk=None, ws=None)
    assert lib.qk_norm_rope_bwd(*{**QK_BWD, **none}.values()) == EUNS          # the rotation alone needs none of these
    assert lib.glu_fwd(*{**GLU_FWD, **dict(a=None, b=None, R=None, GU=None)}.values()) == EUNS
    assert lib.glu_bwd_input(*{**GLU_IN, **dict(p=0.0, dZ=None)}.values()) == EUNS
    assert lib.glu_bwd_weights(*{**GLU_W, **dict(da=None, db=None, scratch=None)}.values()) == EUNS


def test_binding_refuses_wrong_tensors(monkeypatch):
    """Types, shapes, layouts and places, before the library sees a pointer."""
    monkeypatch.setattr(mlp, "_device", lambda: 0)
    bf = dict(dtype=torch.bfloat16)
    T, h, f = 4, 16, 24
    good = dict(X=torch.zeros(T, h, **bf), A=torch.zeros(h, 2 * f, **bf), a=None, B=torch.zeros(f, h, **bf), b=None, R=None, GU=None,
                Y=torch.zeros(T, f, **bf), O=torch.zeros(T, h, **bf))
    for k, v in (("A", torch.zeros(h, f, **bf)), ("X", torch.zeros(T, h)), ("Y", None), ("B", torch.zeros(h, f, **bf)),
                 ("GU", torch.zeros(T, f, **bf)), ("a", torch.zeros(f, **bf))):
        with pytest.raises(ValueError):
            mlp.glu_fwd(h, f, 1, T, 0.0, 1, 0, mlp.GLU_SILU, **{**good, k: v})
    with pytest.raises(ValueError, match="CUDA"):       # a host tensor of the right shape
        mlp.glu_fwd(h, f, 1, T, 0.0, 1, 0, mlp.GLU_SILU, **good)
    Q = torch.zeros(T, 2, 16, **bf)
    pos, inv = torch.zeros(1, T, dtype=torch.int32), torch.zeros(8)
    for q, qo in ((Q.float(), Q), (Q, torch.zeros(T, 3, 16, **bf)), (Q.transpose(0, 1), Q)):
        with pytest.raises(ValueError):
            mlp.qk_norm_rope_fwd(q, Q, qo, Q, pos, inv)
    with pytest.raises(ValueError):
        mlp._rope_args(T, 16, pos, inv, None, None, None, [2, 2, 2, 2], False, 1e-6, 0)
    with pytest.raises(ValueError):
        mlp._rope_args(T, 16, pos.long(), inv, None, None, None, None, False, 1e-6, 0)


class _Fake:
    """A tensor of another device, for machines without one."""
    dtype, is_cuda, device = torch.bfloat16, True, torch.device("cuda", 1)

    def __init__(self, *shape, strides=None):
        self.shape, self.strides = torch.Size(shape), strides

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def stride(self):
        return self.strides

    def data_ptr(self):
        return GOOD


def test_binding_refuses_another_device_and_other_strides():
    """A tensor of a device that is not the current one is refused: the launch would go to the current one's stream."""
    with pytest.raises(ValueError, match="current device"):
        mlp._arg("X", _Fake(4, 16), torch.bfloat16, (4, 16), 0)
    with pytest.raises(ValueError, match="current device"):
        mlp._rows("Q", _Fake(4, 2, 16, strides=(32, 16, 1)), (4, 2, 16), 0)
    assert mlp._rows("Q", _Fake(4, 2, 16, strides=(96, 16, 1)), (4, 2, 16), 1) == (GOOD, 96)
    assert mlp._rows("Q", _Fake(1, 2, 16, strides=(7, 16, 1)), (1, 2, 16), 1) == (GOOD, 32)   # one row: no stride
    for strides in ((96, 48, 1), (96, 16, 2), (1, 4, 8)):
        with pytest.raises(ValueError, match="side by side"):
            mlp._rows("Q", _Fake(4, 2, 16, strides=strides), (4, 2, 16), 1)


def test_workspace_size_matches_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gb_mlp.h")).read()
    rows = int(re.search(r"#define QK_NORM_ROPE_WS_ROWS (\d+)", text).group(1))
    assert mlp.qk_norm_rope_workspace(128) == rows * 2 * 128
