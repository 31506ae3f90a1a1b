"""Refusals of the binding that go wrong before a tensor is looked at."""
import types

import pytest
import torch

from transformer_lm_megatron_gb300 import mlp


@pytest.mark.parametrize("tokens,seq_len", [(64, 0), (64, -8), (60, 32)])
def test_attn_rope_refuses_a_sequence_length(tokens, seq_len, monkeypatch):
    monkeypatch.setattr(mlp, "_device", lambda: 0)
    rope = types.SimpleNamespace()
    with pytest.raises(ValueError, match="seq_len"):
        mlp.attn_rope_fwd(256, 4, 1, tokens, seq_len, 0.1, 1, 0, rope, *[None] * 12)
    with pytest.raises(ValueError, match="seq_len"):
        mlp.attn_rope_bwd(256, 4, 1, tokens, seq_len, 0.1, 1, 0, rope, 1, 0, *[None] * 18)


def test_qk_norm_rope_refuses_missing_tensors(monkeypatch):
    monkeypatch.setattr(mlp, "_device", lambda: 0)
    x = torch.zeros(4, 2, 16, dtype=torch.bfloat16)
    for q, k in ((None, x), (x, None)):
        with pytest.raises(ValueError, match="missing"):
            mlp.qk_norm_rope_fwd(q, k, x, x, None, None)
        with pytest.raises(ValueError, match="missing"):
            mlp.qk_norm_rope_bwd(x, x, q, k, x, x, None, None)
