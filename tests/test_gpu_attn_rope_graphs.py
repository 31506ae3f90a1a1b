"""The attention block with head norms and rotation captured into graphs.

Two graphs captured on one stream are replayed at once on two others: each gives the bits that it gives
alone, and that the eager call gives without the split tail (the order of the tiles changes no bit).  The
shape is one whose eager products use the stream's static workspaces: the 105 tiles of the QKV projection
leave 29 for a second wave of 76 pairs, the 35 tiles of the output projection are less than half of one,
both of 20 k-blocks, and dQ is 140 tiles of one batched product.
"""
import pytest
import torch

import test_gpu_decoder_layer as layer
from transformer_lm_megatron_gb300 import build as gb_build
from transformer_lm_megatron_gb300 import mlp

pytestmark = pytest.mark.gpu

T, H, HEADS, L = 1792, 1280, 20, 256
OUT = ("QKV", "P", "O", "out", "dQKV", "dX", "dWqkv", "dbqkv", "dWo", "dbo")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gb_build.build()
    mlp.load()


@pytest.fixture
def attn_core(request):
    mlp.mlp_set_attn_fused(request.param == "fused")
    yield request.param
    mlp.mlp_set_attn_fused(True)
    mlp.mlp_set_split_tail(True)


def _outputs(y):
    return {**{n: getattr(y.buf, n).clone() for n in OUT}, "QKr": y.QKr.clone(), "dwq": y.rope.dwq.clone(), "dwk": y.rope.dwk.clone()}


@pytest.mark.parametrize("attn_core", ["fused", "unfused"], indirect=True)
def test_graphs_captured_on_one_stream_run_at_once(attn_core):
    ys, ins = [], []
    for seed in (3, 4):
        ys.append(layer.Layer(T, H, HEADS, L, 64, False, [32], True, seed=seed))
        g = torch.Generator().manual_seed(seed)
        ins.append(tuple(layer._randn(g, T, H).cuda() for _ in range(2)))
    one, graphs = torch.cuda.Stream(), []
    for y, (X, dOut) in zip(ys, ins):
        y.fwd(X)
        y.bwd(X, dOut)
        layer._status_ok()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=one):
            y.fwd(X)
            y.bwd(X, dOut)
        graphs.append(g)
    mlp.mlp_set_split_tail(False)
    ref = []
    for y, (X, dOut) in zip(ys, ins):
        y.fwd(X)
        y.bwd(X, dOut)
        layer._status_ok()
        ref.append(_outputs(y))
    mlp.mlp_set_split_tail(True)
    for y, g, r in zip(ys, graphs, ref):
        g.replay()
        layer._status_ok()
        for n, v in _outputs(y).items():
            assert torch.equal(v, r[n]), n
    streams = [torch.cuda.Stream() for _ in ys]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    layer._status_ok()
    for y, r in zip(ys, ref):
        for n, v in _outputs(y).items():
            assert torch.equal(v, r[n]), n
