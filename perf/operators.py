"""Measured cases of the gated feed-forward block and of the head norms with position rotation.

Gated feed-forward block (the MLP block with a gate; act is SiLU or the tanh form of GeLU):
    G = X Ag + ag,  U = X Au + au,  Y = act(G) * U,  O = R + dropout(Y B + b)
    A = [Ag | Au] [h, 2 ffn], GU = [G | U] [tokens, 2 ffn]; the residual R is X.
  glu_fwd          O, and for training the stored GU and Y (bf16)
  glu_bwd_input    dZ = dO * keep / (1 - p), dGU = [dY U act'(G) | dY act(G)] with dY = dZ B^T,
                   dX = dO + dGU A^T, from the stored GU
  glu_bwd_weights  dA = X^T dGU, da = sum dGU, dB = Y^T dZ, db = sum dZ in fp32, from the stored
                   tensors (a pass of its own, so that a pipeline stage can send dX first)
Norms of queries and keys for each head, with the rotation by (one, two or three axes of) positions:
    n = x * rsqrt(mean(x^2) + eps) * w  (or n = x without weights);  each pair (n_i, n_j) of the first `rot`
    dimensions turns by the angle position[axis(i)] * inv_freq[i]
  qk_norm_rope_fwd, qk_norm_rope_bwd (dx for queries and keys, dw in fp32).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
SEED, TOKEN_OFFSET = 1234, 4096
M64 = (1 << 64) - 1


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one sequence through the block of the mid workload (h 4096, ffn 16384): all weights for one row
        dict(name="glu_fwd_one_token", op="glu_fwd", tokens=1, h=4096, ffn=16384, act="silu", p=0.0, bias=False, save=False),
        # a batch of sequences, one token each; ffn is no multiple of any tile
        dict(name="glu_fwd_batch_of_tokens", op="glu_fwd", tokens=27, h=2048, ffn=5464, act="silu", p=0.0, bias=True, save=False),
        # training on a ragged batch, with biases, dropout and the GeLU gate
        dict(name="glu_fwd_train_ragged", op="glu_fwd", tokens=1317, h=1032, ffn=2744, act="gelu", p=0.1, bias=True, save=True),
        # training at the widths of the accumulation sweep (h 8192, ffn 32768): the largest
        dict(name="glu_fwd_train_wide", op="glu_fwd", tokens=2048, h=8192, ffn=32768, act="silu", p=0.0, bias=False, save=True),
        # input gradient of the mid workload
        dict(name="glu_bwd_input_mid", op="glu_bwd_input", tokens=2048, h=4096, ffn=16384, act="silu", p=0.0, bias=False, save=True),
        # the same of the ragged batch, with dropout
        dict(name="glu_bwd_input_ragged", op="glu_bwd_input", tokens=1317, h=1032, ffn=2744, act="gelu", p=0.1, bias=True, save=True),
        # weight gradients of the mid workload, without biases
        dict(name="glu_bwd_weights_mid", op="glu_bwd_weights", tokens=2048, h=4096, ffn=16384, act="silu", p=0.0, bias=False, save=True),
        # weight and bias gradients of the ragged batch
        dict(name="glu_bwd_weights_ragged", op="glu_bwd_weights", tokens=1317, h=1032, ffn=2744, act="gelu", p=0.1, bias=True, save=True),
        # one token far into its sequence, four query heads to a key head: latency
        dict(name="qk_fwd_one_token", op="qk_fwd", tokens=1, nq=32, nk=8, d=128, rot=128, pairs="half", axes=1, norm=True, far=1000000),
        # a whole sequence at the MT-NLG layer's heads (128 of size 160), read out of the fused QKV projection
        dict(name="qk_fwd_mtnlg_heads", op="qk_fwd", tokens=2048, nq=128, nk=128, d=160, rot=160, pairs="half", axes=1, norm=True, far=0),
        # training on video patches: three axes of positions, an odd number of tokens
        dict(name="qk_bwd_three_axes", op="qk_bwd", tokens=8209, nq=32, nk=8, d=128, rot=128, pairs="half", axes=3, norm=True, far=0),
        # part of each head turned, neighbouring pairs, no norm: the rotation alone and its backward
        dict(name="qk_bwd_rotation_only", op="qk_bwd", tokens=3001, nq=16, nk=16, d=80, rot=48, pairs="neighbours", axes=2, norm=False, far=0),
    ]


def _flops(c):
    per = 3 * c["tokens"] * c["h"] * c["ffn"]
    return 2.0 * per


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    most = 3 * 2 * 2048 * 8192 * 32768
    op = rng.choice(["glu_fwd", "glu_fwd", "glu_bwd_input", "glu_bwd_weights", "qk_fwd", "qk_bwd"])
    if op.startswith("glu"):
        while True:
            tokens = _log(rng, 1, 300) if op == "glu_fwd" and rng.random() < 0.5 else _log(rng, 33, 4096)
            h, ffn = _log(rng, 256, 8192, 8), _log(rng, 512, 32768, 8)
            c = dict(op=op, tokens=tokens, h=h, ffn=ffn, act=rng.choice(["silu", "gelu"]), p=rng.choice([0.0, 0.1]),
                     bias=rng.random() < 0.5, save=op != "glu_fwd" or tokens > 300 or rng.random() < 0.3)
            if _flops(c) <= most / 8:
                return c
    d = rng.choice([32, 64, 72, 80, 96, 128, 160, 192, 256])
    rot = rng.choice([d, d, d, 8 * rng.randint(2, d // 8)])
    nk = rng.choice([1, 2, 4, 8, 16, 24, 32])
    nq = nk * rng.choice([1, 2, 4, 5, 8])
    tokens = _log(rng, 1, max(1, min(20000, 100000000 // ((nq + nk) * d))))
    return dict(op=op, tokens=tokens, nq=nq, nk=nk, d=d, rot=rot, pairs=rng.choice(["half", "neighbours"]), axes=rng.choice([1, 1, 2, 3]),
                norm=rng.random() < 0.7, far=rng.choice([0, 0, 120000, 4000000]))


def work(case):
    c = case
    if c["op"].startswith("qk"):
        n = c["tokens"] * (c["nq"] + c["nk"]) * c["d"]
        small = 4 * c["tokens"] * c["axes"] + 2 * c["rot"]
        if c["op"] == "qk_fwd":
            return {"bytes": 4 * n + small + 4 * c["d"] * c["norm"], "flops": (3 + 4 * c["norm"]) * n}
        return {"bytes": (4 + 2 * c["norm"]) * n + small + 12 * c["d"] * c["norm"], "flops": (3 + 12 * c["norm"]) * n}
    T, h, f = c["tokens"], c["h"], c["ffn"]
    weights, both = 2 * 3 * h * f, 2 * (2 * f + h) if c["bias"] else 0
    if c["op"] == "glu_fwd":
        by = weights + both + 2 * T * h * 2 + (2 * T * 3 * f if c["save"] else 0)
    elif c["op"] == "glu_bwd_input":
        by = weights + 2 * T * h * (2 + (c["p"] > 0)) + 2 * T * 4 * f
    else:
        by = 2 * weights + 2 * both + 2 * T * (2 * h + 3 * f)
    return {"bytes": by, "flops": _flops(c)}


# ------------------------------------------------------------------------------------------ the inputs
def _sections(c):
    """Pairs of each axis: as even as they can be, the rest with the first."""
    n = c["rot"] // 2
    each = n // c["axes"]
    return [n - each * (c["axes"] - 1)] + [each] * (c["axes"] - 1)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=g, device=dev).mul_(std).to(torch.bfloat16)  # noqa: E731
    s = dict(c)
    bf = lambda *n: torch.empty(n, dtype=torch.bfloat16, device=dev)  # noqa: E731
    f32 = lambda *n: torch.empty(n, dtype=torch.float32, device=dev)  # noqa: E731
    T = c["tokens"]
    if c["op"].startswith("glu"):
        h, f = c["h"], c["ffn"]
        std = 0.02
        if c["op"] != "glu_bwd_weights":
            s["A"], s["B"] = rnd(h, 2 * f, std=std), rnd(f, h, std=std)
            s["a"], s["b"] = (rnd(2 * f, std=std), rnd(h, std=std)) if c["bias"] else (None, None)
        if c["op"] == "glu_fwd":
            s["X"] = rnd(T, h)
            s["GU"], s["Y"], s["O"] = bf(T, 2 * f) if c["save"] else None, bf(T, f), bf(T, h)
            return s
        s["GU"] = rnd(T, 2 * f, std=std * math.sqrt(h))
        if c["op"] == "glu_bwd_input":
            s["dO"] = rnd(T, h)
            s["dZ"], s["dGU"], s["dX"] = bf(T, h) if c["p"] > 0 else None, bf(T, 2 * f), bf(T, h)
            return s
        s["X"], s["dZ"], s["dGU"] = rnd(T, h), rnd(T, h), rnd(T, 2 * f)
        if c["p"] > 0:
            s["dZ"] *= torch.rand(T, h, generator=g, device=dev) >= c["p"]
        u = s["GU"].float()
        s["Y"] = (u[:, :f].sigmoid() * u[:, :f] * u[:, f:]).to(torch.bfloat16)
        del s["GU"]
        s["dA"], s["dB"] = f32(h, 2 * f), f32(f, h)
        s["da"], s["db"] = (f32(2 * f), f32(h)) if c["bias"] else (None, None)
        s["scratch"] = f32(T, h)
        return s
    nq, nk, d, rot = c["nq"], c["nk"], c["d"], c["rot"]
    # queries and keys side by side with the values in one projection's output, as a block has them
    QKV = rnd(T, (nq + 2 * nk) * d, std=1.5)
    s["Q"], s["K"] = QKV[:, : nq * d].view(T, nq, d), QKV[:, nq * d : (nq + nk) * d].view(T, nk, d)
    pos = torch.arange(T, device=dev, dtype=torch.int32) + c["far"]
    if c["axes"] > 1:
        w = max(1, int(math.sqrt(T / 4)))
        cut = [pos // (w * w), pos // w % w, pos % w]
        s["pos"] = torch.stack(cut[3 - c["axes"] :]).contiguous()
    else:
        s["pos"] = pos[None].contiguous()
    s["pos"] += int(torch.randint(0, 512, (1,), generator=g, device=dev))
    s["sections"] = _sections(c)
    s["axis"] = torch.cat([torch.full((n,), k, device=dev) for k, n in enumerate(s["sections"])])
    # each axis has its own falling frequencies
    s["inv_freq"] = torch.cat([10000.0 ** (-torch.arange(n, device=dev, dtype=torch.float64) / n) for n in s["sections"]]).float()
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2)) if c["norm"] else (None, None)
    if c["op"] == "qk_fwd":
        s["Qo"], s["Ko"] = bf(T, nq, d), bf(T, nk, d)
        return s
    s["dQo"], s["dKo"] = rnd(T, nq, d), rnd(T, nk, d)
    dQKV = bf(T, (nq + 2 * nk) * d)
    s["dQ"], s["dK"] = dQKV[:, : nq * d].view(T, nq, d), dQKV[:, nq * d : (nq + nk) * d].view(T, nk, d)
    s["dwq"], s["dwk"] = (f32(d), f32(d)) if c["norm"] else (None, None)
    s["ws"] = f32(2048 * d) if c["norm"] else None
    return s


# ------------------------------------------------------------------------------------------ the plain forms
def _keep(T, h, p):
    """The block's keep mask: the high 32 bits of output (offset + token) h + column of a SplitMix64 stream against p."""
    e = torch.arange(TOKEN_OFFSET * h, (TOKEN_OFFSET + T) * h, device="cuda", dtype=torch.int64)
    s64 = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
    shr = lambda z, n: (z >> n) & ((1 << (64 - n)) - 1)  # noqa: E731
    z = (e + 1) * s64(0x9E3779B97F4A7C15) + SEED
    z = (z ^ shr(z, 30)) * s64(0xBF58476D1CE4E5B9)
    z = (z ^ shr(z, 27)) * s64(0x94D049BB133111EB)
    z = z ^ shr(z, 31)
    return (shr(z, 32) >= int(math.floor(float(np.float32(p)) * 2**32 + 0.5))).view(T, h)


def _scale(p):
    return float(np.float32(1) / (np.float32(1) - np.float32(p)))


def _act(g, act):
    """act(g) and act'(g)."""
    if act == "silu":
        r = torch.sigmoid(g)
        return g * r, r * (1 + g * (1 - r))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _glu_fwd(s):
    f, T, h = s["ffn"], s["tokens"], s["h"]
    X = s["X"].float()
    GU = X @ s["A"].float()
    if s["a"] is not None:
        GU += s["a"].float()
    Y = _act(GU[:, :f], s["act"])[0] * GU[:, f:]
    Z = Y @ s["B"].float()
    if s["b"] is not None:
        Z += s["b"].float()
    if s["p"] > 0:
        Z = torch.where(_keep(T, h, s["p"]), Z * _scale(s["p"]), 0.0)
    O = (X + Z).bfloat16()
    return [O, GU.bfloat16(), Y.bfloat16()] if s["save"] else [O]


def _glu_bwd_input(s):
    f, T, h = s["ffn"], s["tokens"], s["h"]
    dO = s["dO"].float()
    dZ = torch.where(_keep(T, h, s["p"]), dO * _scale(s["p"]), 0.0) if s["p"] > 0 else dO
    dY = dZ @ s["B"].float().t()
    G, U = s["GU"][:, :f].float(), s["GU"][:, f:].float()
    y, dy = _act(G, s["act"])
    dGU = torch.cat([dY * U * dy, dY * y], 1)
    dX = (dO + dGU @ s["A"].float().t()).bfloat16()
    return [dX, dGU.bfloat16()] + ([dZ.bfloat16()] if s["p"] > 0 else [])


def _glu_bwd_weights(s):
    X, dZ, dGU, Y = (s[k].float() for k in ("X", "dZ", "dGU", "Y"))
    got = [X.t() @ dGU, Y.t() @ dZ]
    if s["bias"]:
        got += [dGU.double().sum(0).float(), dZ.double().sum(0).float()]
    return got


def _angles(s):
    """[tokens, 1, rot / 2] cosines and sines, the angles in 64 bits."""
    a = s["pos"].double().t()[:, s["axis"]] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, s):
    """Each pair of the first rot dimensions by its angle."""
    r, rest = x[..., : s["rot"]], x[..., s["rot"] :]
    if s["pairs"] == "half":
        a, b = r[..., : s["rot"] // 2], r[..., s["rot"] // 2 :]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _qk_fwd(s):
    cos, sin = _angles(s)
    got = []
    for x, w in ((s["Q"], s["wq"]), (s["K"], s["wk"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        got.append(_turn(x, cos, sin, s).bfloat16())
    return got


def _qk_bwd(s):
    cos, sin = _angles(s)
    got, dws = [], []
    for x, w, dy in ((s["Q"], s["wq"], s["dQo"]), (s["K"], s["wk"], s["dKo"])):
        g = _turn(dy.float(), cos, -sin, s)
        if w is not None:
            x = x.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            n = x * r
            dws.append((g * n).sum(1).double().sum(0).float())
            g = g * w.float()
            g = r * (g - n * (g * n).mean(-1, keepdim=True))
        got.append(g.bfloat16())
    return got + dws


PLAIN = {"glu_fwd": _glu_fwd, "glu_bwd_input": _glu_bwd_input, "glu_bwd_weights": _glu_bwd_weights, "qk_fwd": _qk_fwd, "qk_bwd": _qk_bwd}


# ------------------------------------------------------------------------------------------ the framework's calls
def _own(s):
    from transformer_lm_megatron_gb300 import mlp

    op = s["op"]
    if op.startswith("glu"):
        h, f, T, p = s["h"], s["ffn"], s["tokens"], s["p"]
        act = mlp.GLU_SILU if s["act"] == "silu" else mlp.GLU_GELU
    if op == "glu_fwd":
        mlp.glu_fwd(h, f, 1, T, p, SEED, TOKEN_OFFSET, act, s["X"], s["A"], s["a"], s["B"], s["b"], None, s["GU"], s["Y"], s["O"])
        return [s["O"], s["GU"], s["Y"]] if s["save"] else [s["O"]]
    if op == "glu_bwd_input":
        mlp.glu_bwd_input(h, f, 1, T, p, SEED, TOKEN_OFFSET, act, 1, s["dO"], s["A"], s["B"], s["GU"], s["dZ"], s["dGU"], s["dX"])
        return [s["dX"], s["dGU"]] + ([s["dZ"]] if p > 0 else [])
    if op == "glu_bwd_weights":
        mlp.glu_bwd_weights(h, f, 1, T, 0, s["X"], s["dZ"], s["Y"], s["dGU"], s["dA"], s["da"], s["dB"], s["db"], s["scratch"])
        return [s["dA"], s["dB"]] + ([s["da"], s["db"]] if s["bias"] else [])
    kw = dict(wq=s["wq"], wk=s["wk"], eps=EPS, rot=s["rot"], sections=s["sections"], interleaved=s["pairs"] == "neighbours")
    if op == "qk_fwd":
        mlp.qk_norm_rope_fwd(s["Q"], s["K"], s["Qo"], s["Ko"], s["pos"], s["inv_freq"], **kw)
        return [s["Qo"], s["Ko"]]
    mlp.qk_norm_rope_bwd(s["Q"], s["K"], s["dQo"], s["dKo"], s["dQ"], s["dK"], s["pos"], s["inv_freq"], dwq=s["dwq"], dwk=s["dwk"],
                         ws=s["ws"], accumulate=False, **kw)
    return [s["dQ"], s["dK"]] + ([s["dwq"], s["dwk"]] if s["norm"] else [])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------ in 64 bits
def _exact_keep(T, h, p):
    e = np.arange(TOKEN_OFFSET * h + 1, (TOKEN_OFFSET + T) * h + 1, dtype=np.uint64)
    with np.errstate(over="ignore"):
        z = np.uint64(SEED) + e * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    z ^= z >> np.uint64(31)
    keep = (z >> np.uint64(32)) >= np.uint64(round(float(np.float32(p)) * 4294967296))
    return torch.from_numpy(keep.reshape(T, h)).cuda()


def _exact_gate(G, act):
    """The gate's value and slope, from the logistic function alone."""
    if act == "silu":
        v, dv = G, torch.ones_like(G)
    else:  # 0.5 (1 + tanh(v)) is the logistic function of 2 v
        k = 2 * math.sqrt(2 / math.pi)
        v, dv = k * (G + 0.044715 * G**3), k * (1 + 0.134145 * G**2)
    q = 1 / (1 + torch.exp(-v))
    return G * q, q + G * q * (1 - q) * dv


def exact(case, seed):
    s = prepare(case, seed)
    D = lambda k: None if s[k] is None else s[k].double()  # noqa: E731
    if case["op"].startswith("glu"):
        T, h, f, p = s["tokens"], s["h"], s["ffn"], s["p"]
        if case["op"] == "glu_bwd_weights":
            X, dZ, dGU, Y = D("X"), D("dZ"), D("dGU"), D("Y")
            got = [torch.einsum("ti,tj->ij", X, dGU), torch.einsum("ti,tj->ij", Y, dZ)]
            return got + ([dGU.sum(0), dZ.sum(0)] if s["bias"] else [])
        mask = _exact_keep(T, h, p).double() / (1 - float(np.float32(p))) if p > 0 else 1.0
        A, B = D("A"), D("B")
        if case["op"] == "glu_fwd":
            X = D("X")
            G, U = X @ A[:, :f], X @ A[:, f:]
            if s["bias"]:
                G, U = G + D("a")[:f], U + D("a")[f:]
            Y = _exact_gate(G, s["act"])[0] * U
            Z = Y @ B + (D("b") if s["bias"] else 0.0)
            O = X + Z * mask
            return [O, torch.cat([G, U], 1), Y] if s["save"] else [O]
        dO, G, U = D("dO"), D("GU")[:, :f], D("GU")[:, f:]
        dZ = dO * mask
        dY = torch.einsum("th,fh->tf", dZ, B)
        y, slope = _exact_gate(G, s["act"])
        dG, dU = dY * U * slope, dY * y
        dX = dO + torch.einsum("tf,hf->th", dG, A[:, :f]) + torch.einsum("tf,hf->th", dU, A[:, f:])
        return [dX, torch.cat([dG, dU], 1)] + ([dZ] if p > 0 else [])
    T, d, rot = s["tokens"], s["d"], s["rot"]
    # each turned pair as one complex number, multiplied by exp(i angle)
    start = np.cumsum([0] + s["sections"])
    ang = torch.cat([s["pos"][k].double()[:, None] * s["inv_freq"].double()[None, start[k] : start[k + 1]] for k in range(s["axes"])], 1)
    unit = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    i = torch.arange(rot // 2, device="cuda")
    first, second = (i, i + rot // 2) if s["pairs"] == "half" else (2 * i, 2 * i + 1)

    def turned(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "qk_fwd":
        got = []
        for x, w in ((D("Q"), D("wq")), (D("K"), D("wk"))):
            n = x if w is None else x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w
            got.append(turned(n, unit))
        return got
    got, dws = [], []
    for x, w, dy in ((D("Q"), D("wq"), D("dQo")), (D("K"), D("wk"), D("dKo"))):
        g = turned(dy, unit.conj())
        if w is None:
            got.append(g)
            continue
        rms = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
        dws.append((g * x / rms).sum((0, 1)))
        wg = w * g
        got.append(wg / rms - x * (wg * x).sum(-1, keepdim=True) / (d * rms**3))
    return got + dws
