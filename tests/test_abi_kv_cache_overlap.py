"""Refusals of arrays of the key/value cache's calls that lie over one another, before anything touches a device."""
import itertools

import pytest
import torch

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_abi_kv_cache import ATTN, PLAN, _refuse


@pytest.fixture(scope="module")
def lib():
    gb_build.build()
    return mlp.load()


@pytest.mark.parametrize("a,b", list(itertools.combinations(["table", "lens_out", "taken_out", "cu", "pos", "slots", "status"], 2)))
def test_plan_outputs_lie_apart(lib, a, b):
    """Of two arrays, one in the other's last element."""
    words = dict(table=PLAN["n"] * PLAN["width"], lens_out=PLAN["n"], taken_out=1, cu=PLAN["n"] + 1, pos=PLAN["rows"], slots=PLAN["rows"],
                 status=1)
    for x, y in ((a, b), (b, a)):
        _refuse(lib, "kv_plan", PLAN, {x: PLAN[y] + 4 * (words[y] - 1)}, mlp.MLP_EINVAL)


Q, WIDE = ATTN["Q"], ATTN["nq"] * ATTN["d"]  # 16 rows of 256 elements


@pytest.mark.parametrize("kw", [
    dict(O=Q + 16), dict(O=Q - 16), dict(O=Q + 2 * (15 * 256 + 248)), dict(O=Q - 2 * (15 * 256 + 248)),  # dense, by 8 elements at least
    dict(ldq=768, ldo=768, O=Q + 2 * 248), dict(ldq=768, ldo=768, O=Q + 2 * 520), dict(ldq=768, ldo=768, O=Q - 2 * 248),  # slices that meet
    dict(ldq=768, ldo=768, O=Q + 2 * (768 * 15 + 248)), dict(ldq=512, ldo=768, O=Q + 2 * 512), dict(ldq=264, ldo=264, O=Q + 2 * 264)])
def test_attn_output_over_queries(lib, kw):
    _refuse(lib, "kv_attn", ATTN, kw, mlp.MLP_EINVAL)


@pytest.mark.parametrize("kw", [
    dict(O=Q + 2 * 16 * WIDE), dict(O=Q - 2 * 16 * WIDE), dict(ldq=512, ldo=512, O=Q + 2 * 256), dict(ldq=512, ldo=512, O=Q - 2 * 256),
    dict(ldq=776, ldo=776, O=Q + 2 * (776 + 264)), dict(ldq=1024, ldo=512, O=Q + 2 * 256), dict(rows=1, ldq=8192, ldo=256, O=Q + 512)])
def test_attn_output_beside_queries(lib, kw):
    """Behind them, or between them in rows of one buffer: taken (and refused only for want of a device)."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are no device's")
    assert lib.kv_attn(*{**ATTN, **kw}.values()) == mlp.MLP_EUNSUPPORTED
