"""Refusals of the key/value cache's entry points, through the C ABI and the binding, before anything touches a device."""
import os
import re

import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

EINVAL, EALIGN, EUNS = mlp.MLP_EINVAL, mlp.MLP_EALIGN, mlp.MLP_EUNSUPPORTED
P = 1 << 20  # aligned fake addresses, far enough apart: validation fails before anything reads them


@pytest.fixture(scope="module")
def lib():
    gb_build.build()
    return mlp.load()


def _places(*names):
    return {k: P * (i + 1) for i, k in enumerate(names)}


PLAN = dict(n=4, bs=16, width=8, n_free=100, rows=64, **_places("add", "lens", "table", "free", "taken", "lens_out", "taken_out", "cu", "pos",
                                                                 "slots", "status"), stream=None)
WRITE = dict(tokens=16, nk=2, d=64, bs=16, blocks=10, K=P, ldk=128, V=2 * P, ldv=128,
             **{k: v + 4 * P for k, v in _places("slots", "Kc", "Vc", "Kmax", "Vmax").items()}, stream=None)
ATTN = dict(n=4, rows=16, nq=4, nk=2, d=64, bs=16, blocks=10, width=8, scale=0.125, Q=P, ldq=256,
            **{k: v + 4 * P for k, v in _places("Kc", "Vc", "Kmax", "Vmax", "table", "lens", "cu").items()}, O=2 * P, ldo=256, ws=3 * P,
            stream=None)


def _refuse(lib, name, base, kw, code):
    args = {**base, **kw}
    assert set(args) == set(base)
    assert getattr(lib, name)(*args.values()) == code
    assert mlp.last_error()


def _bad_pointers(names, align):
    return [({k: None}, EINVAL) for k in names] + [({k: P + align // 2}, EALIGN) for k in names]


BAD_TABLE = [(dict(n=0), EINVAL), (dict(n=4097), EINVAL), (dict(width=0), EINVAL), (dict(width=1 << 27), EINVAL)]
BAD_BS = [(dict(bs=b), EINVAL) for b in (0, 8, 24, 128, -16)]
BAD_CACHE = BAD_BS + [(dict(nk=0), EINVAL), (dict(nk=65537), EINVAL), (dict(d=0), EINVAL), (dict(d=48), EINVAL), (dict(d=288), EUNS),
                      (dict(blocks=0), EINVAL), (dict(blocks=1 << 27), EINVAL)]


@pytest.mark.parametrize("kw,code", BAD_TABLE + BAD_BS + _bad_pointers([k for k, v in PLAN.items() if v and v >= P], 4) + [
    (dict(n_free=0), EINVAL), (dict(rows=0), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(lens_out=PLAN["lens"]), EINVAL),
    (dict(lens_out=PLAN["lens"] + 12), EINVAL), (dict(taken_out=PLAN["taken"]), EINVAL), (dict(slots=PLAN["add"] - 252), EINVAL),
    (dict(free=PLAN["table"] + 4), EINVAL)])
def test_plan(lib, kw, code):
    _refuse(lib, "kv_plan", PLAN, kw, code)


@pytest.mark.parametrize("kw,code", BAD_CACHE + _bad_pointers(("K", "V", "Kc", "Vc"), 16) + _bad_pointers(("slots", "Kmax", "Vmax"), 4) + [
    (dict(tokens=0), EINVAL), (dict(tokens=1 << 31), EINVAL), (dict(ldk=120), EINVAL), (dict(ldv=132), EINVAL),
    (dict(tokens=(1 << 31) - 1, nk=65536, ldk=65536 * 64, ldv=65536 * 64), EUNS)])
def test_write(lib, kw, code):
    if code == EUNS and "tokens" in kw and not torch.cuda.is_available():
        pytest.skip("found out on the device")
    _refuse(lib, "kv_write", WRITE, kw, code)


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_TABLE + _bad_pointers(("Q", "O", "Kc", "Vc", "ws"), 16)
                         + _bad_pointers(("Kmax", "Vmax", "table", "lens", "cu"), 4) + [
    (dict(nq=0), EINVAL), (dict(nq=3), EINVAL), (dict(nq=131072), EINVAL), (dict(rows=0), EINVAL), (dict(rows=1 << 30), EINVAL),
    (dict(ldq=248), EINVAL), (dict(ldo=260), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(O=P), EINVAL)])
def test_attn(lib, kw, code):
    _refuse(lib, "kv_attn", ATTN, kw, code)


def test_valid_calls_without_a_gpu_report_unsupported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, base in (("kv_plan", PLAN), ("kv_write", WRITE), ("kv_attn", ATTN)):
        assert getattr(lib, name)(*base.values()) == EUNS, name


def test_binding_refuses_wrong_tensors(monkeypatch):
    """Types, shapes, layouts and places, before the library sees a pointer."""
    monkeypatch.setattr(mlp, "_device", lambda: 0)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    plan = dict(add=i(4), lens=i(4), table=i(4, 8), free_list=i(9), taken=i(1), bs=16, lens_out=i(4), taken_out=i(1), cu=i(5), pos=i(6),
                slots=i(6), status=i(1))
    for k, v in (("lens", i(5)), ("table", i(4)), ("table", i(8, 4).t()), ("cu", i(4)), ("slots", i(7)), ("add", None), ("pos", None),
                 ("free_list", torch.zeros(9)), ("add", i(4).long())):
        with pytest.raises(ValueError):
            mlp.kv_plan(**{**plan, k: v})
    cache = dict(Kc=torch.zeros(10, 2, 16, 64, dtype=torch.int8), Vc=torch.zeros(10, 2, 16, 64, dtype=torch.int8),
                 Kmax=torch.zeros(10, 2), Vmax=torch.zeros(10, 2))
    write = dict(K=bf(5, 2, 64), V=bf(5, 2, 64), slots=i(5), **cache)
    for k, v in (("K", bf(5, 3, 64)), ("K", None), ("V", bf(4, 2, 64)), ("slots", i(6)), ("Kc", None), ("Kc", bf(10, 2, 16, 64)),
                 ("Vc", torch.zeros(10, 16, 2, 64, dtype=torch.int8)), ("Kmax", torch.zeros(10)), ("K", bf(2, 5, 64).transpose(0, 1))):
        with pytest.raises(ValueError):
            mlp.kv_write(**{**write, k: v})
    attn = dict(Q=bf(5, 4, 64), O=bf(5, 4, 64), table=i(3, 8), lens=i(3), cu=i(4), ws=torch.zeros(mlp.kv_attn_workspace(64)), **cache)
    for k, v in (("Q", bf(5, 4, 32)), ("Q", None), ("O", bf(4, 4, 64)), ("table", i(3)), ("lens", i(4)), ("cu", i(3)),
                 ("ws", torch.zeros(100)), ("Vmax", torch.zeros(10, 2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            mlp.kv_attn(**{**attn, k: v})
    for call, args in ((mlp.kv_plan, plan), (mlp.kv_write, write), (mlp.kv_attn, attn)):
        with pytest.raises(ValueError, match="CUDA"):  # host tensors of the right shapes
            call(**args)


def test_workspace_size_matches_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gb_mlp.h")).read()
    rows = int(re.search(r"#define KV_ATTN_WS_ROWS (\d+)", text).group(1))
    for d in (32, 128, 256):
        assert mlp.kv_attn_workspace(d) == rows * (d + 2)
