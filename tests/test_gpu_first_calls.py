"""First calls of a process from two host threads at once.

What a kernel's first launch works out (attributes, how many clusters fit) is written once for the
process.  The threads start every first call together, in shapes that reach each form of the gated
block's products, and the attention block's kernels; what they get has the bits of one thread's calls
made afterwards.  (A torn set-up would show as a failed launch or an unlaunched tile.)
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

FRESH = """
import sys, threading
sys.path.insert(0, "tests")
import torch
import test_gpu_decoder_layer as layer, test_gpu_glu as glu
from transformer_lm_megatron_gb300 import mlp
mlp.load()

# few tokens; 256 x 256 tiles; tiles shared by pairs, forwards and in the weight gradients
SHAPES = [(40, 520, 1096), (700, 520, 1096), (700, 1032, 1544), (1400, 264, 520)]
bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")


class Work:
    def __init__(self, seed):
        self.cases = [glu.Case(*s, "silu", 0.1, True, seed=seed) for s in SHAPES]
        self.y = layer.Layer(256, 256, 4, 128, 64, False, [32], True, seed=seed)
        g = torch.Generator().manual_seed(seed)
        self.X, self.dOut = (layer._randn(g, 256, 256).cuda() for _ in range(2))

    def run(self, start):
        got = []
        for c, (T, h, f) in zip(self.cases, SHAPES):
            GU, Y, O = torch.empty(T, 2 * f, **bf), torch.empty(T, f, **bf), torch.empty(T, h, **bf)
            dZ, dGU, dX = torch.empty(T, h, **bf), torch.empty(T, 2 * f, **bf), torch.empty(T, h, **bf)
            dA, da, dB, db = torch.empty(h, 2 * f, **f32), torch.empty(2 * f, **f32), torch.empty(f, h, **f32), torch.empty(h, **f32)
            start()
            c.fwd(GU, Y, O)
            start()
            c.bwd_input(GU, dZ, dGU, dX)
            start()
            c.bwd_weights(dZ, Y, dGU, dA, da, dB, db)
            got += [GU, Y, O, dZ, dGU, dX, dA, da, dB, db]
        start()
        self.y.fwd(self.X)
        start()
        self.y.bwd(self.X, self.dOut)
        b = self.y.buf
        return got + [t.clone() for t in (b.QKV, b.out, b.dX, b.dWqkv, b.dbqkv, b.dWo, b.dbo, self.y.rope.dwq, self.y.rope.dwk)]


works = [Work(s) for s in (1, 2)]
torch.cuda.synchronize()
barrier = threading.Barrier(2, timeout=120)
outs, errors = {}, []


def thread(w):
    try:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs[w] = w.run(barrier.wait)
        s.synchronize()
    except Exception as e:
        errors.append(repr(e))
        barrier.abort()


threads = [threading.Thread(target=thread, args=(w,)) for w in works]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
glu._status_ok()
for w in works:
    for a, b in zip(outs[w], w.run(lambda: None)):
        assert torch.equal(a, b)
glu._status_ok()
print("first calls agree")
"""


def test_first_calls_from_two_threads():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "agree" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
