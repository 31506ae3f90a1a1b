"""Refusals of arrays of the key/value cache's calls that lie over one another, before anything touches a device."""
import itertools

import pytest

from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

from test_abi_kv_cache import PLAN, _refuse


@pytest.fixture(scope="module")
def lib():
    gb_build.build()
    return mlp.load()


@pytest.mark.parametrize("a,b", itertools.combinations(["table", "lens_out", "taken_out", "cu", "pos", "slots", "status"], 2))
def test_plan_outputs_lie_apart(lib, a, b):
    """Of two arrays, one in the other's last element."""
    words = dict(table=PLAN["n"] * PLAN["width"], lens_out=PLAN["n"], taken_out=1, cu=PLAN["n"] + 1, pos=PLAN["rows"], slots=PLAN["rows"],
                 status=1)
    for x, y in ((a, b), (b, a)):
        _refuse(lib, "kv_plan", PLAN, {x: PLAN[y] + 4 * (words[y] - 1)}, mlp.MLP_EINVAL)
