"""Measured cases of the key/value cache held in 8 bits: its block tables, the write into it, the attention over it.

Blocks of bs tokens; Kc, Vc [blocks, nk, bs, d] int8, Kmax, Vmax [blocks, nk] fp32: a code c stands for c * max / 127.
  kv_plan   from the tokens that n requests hold and get: blocks off a free list into their tables, the offsets of
            their new tokens' rows, and each row's position and slot (block * bs + place in the block)
  kv_write  K, V [tokens, nk, d] bf16 into their slots: max = the largest magnitude of the block's tokens for that
            head, code = rint(x * 127 / max); codes already in the block go from the old max to the new one
  kv_attn   O = softmax(scale Q K^T) V over each request's tokens, its new tokens being the last ones, each of which
            sees itself and what is before it; nq / nk query heads share a key head
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a step of a batch: one new token for each request, a new block for one in sixteen
        dict(name="plan_step", op="plan", n=64, bs=16, most=1, held=4096, pad=0),
        # prompts of ragged lengths come in together; the rows of a fixed-size batch are not all used
        dict(name="plan_prompts", op="plan", n=500, bs=32, most=250, held=0, pad=333),
        # one token of one request: latency
        dict(name="write_one_token", op="write", n=1, most=1, nk=8, d=128, bs=16, held=1000, pad=0),
        # one token for each request of a batch
        dict(name="write_step", op="write", n=130, most=1, nk=8, d=128, bs=32, held=2000, pad=6),
        # ragged prompts
        dict(name="write_prompts", op="write", n=9, most=3001, nk=8, d=128, bs=16, held=0, pad=0),
        # whole sequences at the MT-NLG layer's heads (128 of size 160)
        dict(name="write_mtnlg_heads", op="write", n=2, most=2048, nk=128, d=160, bs=64, held=0, pad=0),
        # one token of one short request: latency
        dict(name="attn_one_short", op="attn", n=1, new=1, nq=32, nk=8, d=128, bs=16, lo=137, hi=137),
        # one token of one long request: the sequence is the only thing to share out
        dict(name="attn_one_long", op="attn", n=1, new=1, nq=32, nk=8, d=128, bs=16, lo=131077, hi=131077),
        # a batch of requests whose lengths differ by two orders of magnitude
        dict(name="attn_ragged", op="attn", n=48, new=1, nq=32, nk=8, d=128, bs=32, lo=100, hi=16384),
        # a full batch of long requests: the largest
        dict(name="attn_batch", op="attn", n=64, new=1, nq=64, nk=8, d=128, bs=64, lo=12000, hi=16384),
        # the MT-NLG layer's heads, each with its own keys
        dict(name="attn_mtnlg_heads", op="attn", n=8, new=1, nq=128, nk=128, d=160, bs=16, lo=1500, hi=2048),
        # five drafted tokens for each request, eight query heads to a key head
        dict(name="attn_drafts", op="attn", n=16, new=5, nq=32, nk=4, d=128, bs=16, lo=3000, hi=9000),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "write", "attn", "attn", "attn"])
    bs, pad = rng.choice([16, 32, 64]), rng.choice([0, 0, 1, 77])
    if op == "plan":
        return dict(op=op, n=_log(rng, 1, 2000), bs=bs, most=_log(rng, 1, 300), held=rng.choice([0, 100, 5000]), pad=pad)
    d = 32 * rng.randint(1, 8)
    nk = rng.choice([1, 2, 3, 4, 8, 16, 32, 64])
    if op == "write":
        n, most = _log(rng, 1, 300), rng.choice([1, 1, 5, _log(rng, 1, 4000)])
        while n * most * nk * d > 90000000:
            most, n = max(1, most // 2), max(1, n // 2)
        return dict(op=op, n=n, most=most, nk=nk, d=d, bs=bs, held=rng.choice([0, 17, 3000]), pad=pad)
    new = rng.choice([1, 1, 1, 2, 3, 4, 7])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16])
    n, hi = _log(rng, 1, 128), _log(rng, 20, 200000)
    while n * hi * nk * d > 64 * 16384 * 8 * 128 // 2 or n * hi * nk * group * new > 40000000:
        n, hi = max(1, n * 2 // 3), max(20, hi * 2 // 3)
        nk = max(1, nk // 2) if n == 1 and hi < 1000 else nk
    return dict(op=op, n=n, new=new, nq=nk * group, nk=nk, d=d, bs=bs, lo=max(new, _log(rng, 1, hi)), hi=hi)


def _lengths(c):
    """The tokens that each request gets (plan, write) or has (attn); the same for every seed, so that work() knows them."""
    u = _uniform(c, 0)
    if c["op"] == "attn":
        return (math.log(c["lo"]) + u * math.log(c["hi"] / c["lo"])).exp().round().long().clamp(c["lo"], c["hi"])
    return (u * c["most"]).long() + 1


def _held(c):
    """The tokens that each request has already (plan, write)."""
    return (_uniform(c, 1) * (c["held"] + 1)).long()


def _uniform(c, k):
    g = torch.Generator().manual_seed(c["n"] * 7919 + (c["hi"] if c["op"] == "attn" else c["most"]) + 104729 * k)
    return torch.rand(c["n"], generator=g, dtype=torch.float64)


def work(case):
    c, lens = case, _lengths(case)
    total, n = int(lens.sum()), c["n"]
    if c["op"] == "plan":
        # lengths in and out, offsets; each row's position and slot; a new block's entry in the list and in the table
        return {"bytes": 16 * n + 8 * (total + c["pad"]) + 8 * (total // c["bs"]), "flops": 0}
    rows = 2 * c["nk"] * c["d"]
    if c["op"] == "write":
        blocks = n if c["most"] == 1 else total // c["bs"]
        return {"bytes": total * rows * 3 + 4 * total + blocks * 2 * c["nk"] * 4, "flops": 3 * total * rows}
    held = int(((lens + c["bs"] - 1) // c["bs"]).sum())
    return {"bytes": total * rows + held * (4 + 8 * c["nk"]) + 4 * n * c["new"] * c["nq"] * c["d"], "flops": 4 * total * c["new"] * c["nq"] * c["d"]}


# ------------------------------------------------------------------------------------------ the inputs
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(c)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
    n, bs = c["n"], c["bs"]
    lens = _lengths(c).to(dev, torch.int32)
    held = lens if c["op"] == "attn" else _held(c).to(dev, torch.int32)
    top = int(held.max()) + (0 if c["op"] == "attn" else int(lens.max()))
    width = (top + bs - 1) // bs
    have = (held + bs - 1) // bs
    first = torch.cumsum(have, 0) - have
    at = torch.arange(width, device=dev)
    if c["op"] == "plan":
        blocks = int(have.sum()) + int(((held + lens + bs - 1) // bs - have).sum()) + 5
    elif c["op"] == "write":
        # each request's slots run on from what it holds; only its last blocks matter, so the pool has no others
        blocks = int(((held % bs + lens + bs - 1) // bs).sum()) + 2
    else:
        blocks = int(have.sum()) + 3
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    if c["op"] in ("plan", "attn"):
        ids = order[(first[:, None] + at).clamp(max=blocks - 1)]
        s["table"] = torch.where(at < have[:, None], ids, -1).to(torch.int32).contiguous()
    if c["op"] == "plan":
        s["add"], s["lens"] = lens, held.contiguous()
        s["free"] = torch.cat([order, order[:1]])[: blocks].contiguous()
        s["taken"] = have.sum().to(torch.int32)[None]
        T = int(lens.sum()) + c["pad"]
        s["lens_out"], s["taken_out"], s["cu"], s["status"] = i32(n), i32(1), i32(n + 1), i32(1)
        s["pos"], s["slots"] = i32(T), i32(T)
        return s
    nk, d = c["nk"], c["d"]
    if c["op"] == "write":
        off = held % bs  # of the last block that is not full
        each = (off + lens + bs - 1) // bs
        start = (torch.cumsum(each, 0) - each).long()
        r = torch.repeat_interleave(torch.arange(n, device=dev), lens.long())
        p = torch.arange(r.numel(), device=dev) - (torch.cumsum(lens, 0) - lens).long()[r] + off[r]
        slots = order[start[r] + p // bs].long() * bs + p % bs
        s["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, device=dev)]).to(torch.int32)
        T = s["slots"].numel()
        # keys and values as they lie in a projection's output: a few dimensions are far larger than the others
        wide = 1 + 7 * (torch.rand(2 * nk * d, generator=g, device=dev) < 0.02)
        KV = (torch.randn(T, 2 * nk * d, generator=g, device=dev) * wide).to(torch.bfloat16)
        s["K"], s["V"] = KV[:, : nk * d].view(T, nk, d), KV[:, nk * d :].view(T, nk, d)
    # what the cache holds: codes of normally distributed values, a max for each block and head that bf16 can hold
    for k in ("Kc", "Vc"):
        s[k] = torch.empty(blocks, nk, bs, d, dtype=torch.int8, device=dev)
        s[k].view(-1)[:] = _codes(s[k].numel(), g, dev)
    for k in ("Kmax", "Vmax"):
        s[k] = (3.0 * torch.exp(0.4 * torch.randn(blocks, nk, generator=g, device=dev))).bfloat16().float()
    if c["op"] == "attn":
        T = n * c["new"]
        s["Q"] = torch.randn(T, c["nq"], d, generator=g, device=dev).to(torch.bfloat16)
        s["O"] = torch.zeros_like(s["Q"])
        s["lens"], s["cu"] = lens, torch.arange(n + 1, device=dev, dtype=torch.int32) * c["new"]
        s["ws"] = torch.empty(2 * 9728 * (d + 2), dtype=torch.float32, device=dev)
    return s


def _codes(n, g, dev):
    """n codes in [-127, 127]: a million drawn ones, laid end to end from places of their own."""
    some = (torch.randn(min(n, 1 << 20) + 4099, generator=g, device=dev) * 40).clamp(-127, 127).round().to(torch.int8)
    return some.repeat(-(-n // some.numel()))[:n]


# ------------------------------------------------------------------------------------------ the plain forms
def _plan(s):
    add, old, table, free, bs = s["add"].long(), s["lens"].long(), s["table"], s["free"], s["bs"]
    n, width = table.shape
    have, need = (old + bs - 1) // bs, (old + add + bs - 1) // bs
    cu = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)])
    blocks = torch.cumsum(need - have, 0)
    first, taken = blocks - (need - have), s["taken"].long()
    T = s["slots"].numel()
    # a bit for each reason why the step does not fit: then nothing changes
    status = (taken + blocks[-1:] > free.numel()).int() + 2 * (need > width).any().int() + 4 * (cu[-1:] > T).int()
    status += 8 * ((add < 0) | (old < 0)).any().int()
    fits = status == 0
    cu = torch.where(fits, cu, 0)
    t = torch.arange(T, device=add.device)
    used = t < cu[-1]
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    p = old[r] + t - cu[r]
    b = p // bs
    fresh = free[(taken + first[r] + b - have[r]).clamp(0, free.numel() - 1)]
    block = torch.where(b < have[r], table[r, b.clamp(0, width - 1)], fresh).long()
    slots, pos = torch.where(used, block * bs + p % bs, -1).int(), torch.where(used, p, 0).int()
    # a new block's first token is a new one; what is no such token writes where nothing is read
    cells = torch.cat([table.view(-1), table.new_zeros(1)])
    cells[torch.where(used & (p % bs == 0), r * width + b, n * width)] = block.int()
    table.copy_(cells[:-1].view(n, width))
    return {"lens": (old + fits * add).int(), "taken": (taken + fits * blocks[-1:]).int(), "cu": cu.int(), "pos": pos, "slots": slots,
            "table": table, "status": status.int()}


def _write(s):
    slots, bs, nk = s["slots"].long(), s["bs"], s["nk"]
    T = slots.numel()
    t = torch.arange(T, device=slots.device)
    used = slots >= 0
    before = torch.cat([slots.new_full((1,), -2), slots[:-1]])
    leads = used & ((slots != before + 1) | (slots % bs == 0))
    run = torch.cumsum(leads, 0) - 1  # tokens next to each other in one block
    used = used.nonzero()[:, 0]
    lead = leads.nonzero()[:, 0]
    run, block, off = run[used], slots[used] // bs, slots[used] % bs
    block1, off1 = slots[lead] // bs, slots[lead] % bs  # a run's block, and how many tokens are before it
    heads = torch.arange(nk, device=slots.device)
    for x, codes, most in ((s["K"], s["Kc"], s["Kmax"]), (s["V"], s["Vc"], s["Vmax"])):
        x = x[used].float()
        new = torch.zeros(lead.numel(), nk, device=x.device).scatter_reduce_(0, run[:, None].expand(-1, nk), x.abs().amax(-1), "amax")
        old = torch.where((off1 > 0)[:, None], most[block1], 0.0)
        new = torch.maximum(new, old)
        grown = ((off1 > 0)[:, None] & (new > old)).any(1).nonzero()[:, 0]
        held = codes[block1[grown]].float()
        moved = torch.round(held * old[grown][:, :, None, None] / new[grown][:, :, None, None]).to(torch.int8)
        there = torch.arange(bs, device=x.device) < off1[grown][:, None]
        codes[block1[grown]] = torch.where(there[:, None, :, None], moved, codes[block1[grown]])
        most[block1] = new
        top = new[run][:, :, None]
        codes[block[:, None], heads, off[:, None]] = torch.round(x * 127 / top).to(torch.int8)
    return {k: s[k] for k in ("Kc", "Vc", "Kmax", "Vmax")}


def _attn(s):
    n, new, nq, nk, d, bs = (s[k] for k in ("n", "new", "nq", "nk", "d", "bs"))
    at = s["table"].long().clamp(min=0)
    L = at.shape[1] * bs
    read = lambda codes, most: (codes[at].float() * (most[at] / 127)[..., None, None]).transpose(1, 2).reshape(n, nk, L, d)  # noqa: E731
    q = s["Q"].float().view(n, new, nk, nq // nk, d).permute(0, 2, 1, 3, 4).reshape(n, nk, -1, d)
    x = (q @ read(s["Kc"], s["Kmax"]).transpose(2, 3)).view(n, nk, new, nq // nk, L) * d**-0.5
    last = s["lens"].long()[:, None] - new + torch.arange(new, device=q.device)  # the last token that each one sees
    seen = torch.arange(L, device=q.device) <= last[..., None]
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = (x / x.sum(-1, keepdim=True)).view(n, nk, -1, L)
    o = (x @ read(s["Vc"], s["Vmax"])).view(n, nk, new, nq // nk, d)
    return o.permute(0, 2, 1, 3, 4).reshape(n * new, nq, d).to(torch.bfloat16)


PLAIN = {"plan": _plan, "write": _write, "attn": _attn}


# ------------------------------------------------------------------------------------------ the framework's calls
def _own(s):
    from transformer_lm_megatron_gb300 import mlp

    if s["op"] == "plan":
        mlp.kv_plan(s["add"], s["lens"], s["table"], s["free"], s["taken"], s["bs"], s["lens_out"], s["taken_out"], s["cu"], s["pos"],
                    s["slots"], s["status"])
        return {"lens": s["lens_out"], "taken": s["taken_out"], "cu": s["cu"], "pos": s["pos"], "slots": s["slots"], "table": s["table"],
                "status": s["status"]}
    if s["op"] == "write":
        mlp.kv_write(s["K"], s["V"], s["slots"], s["Kc"], s["Vc"], s["Kmax"], s["Vmax"])
        return {k: s[k] for k in ("Kc", "Vc", "Kmax", "Vmax")}
    mlp.kv_attn(s["Q"], s["Kc"], s["Vc"], s["Kmax"], s["Vmax"], s["table"], s["lens"], s["cu"], s["O"], s["ws"])
    return s["O"]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "write":
        # the largest magnitude of each block, from its tokens one block after another; the codes are whole numbers
        slots, bs = s["slots"].cpu().tolist(), s["bs"]
        tokens = {}
        for t, x in enumerate(slots):
            if x >= 0:
                tokens.setdefault(x // bs, []).append(t)
        got = {"Kc": None, "Vc": None}
        blocks = torch.tensor(list(tokens), device="cuda")
        rows = torch.tensor([v + v[:1] * (bs - len(v)) for v in tokens.values()], device="cuda")
        kept = torch.tensor([slots[v[0]] % bs > 0 for v in tokens.values()], device="cuda")
        for k in ("K", "V"):
            most = s[k + "max"].double()
            seen = torch.stack([s[k][rows[:, j]].double().abs().amax(-1) for j in range(bs)]).amax(0)
            most[blocks] = torch.where(kept[:, None], torch.maximum(seen, most[blocks]), seen)
            got[k + "max"] = most
        return got
    n, new, nq, nk, d, bs = (s[k] for k in ("n", "new", "nq", "nk", "d", "bs"))
    lens, O = s["lens"].tolist(), torch.zeros(n * new, nq, d, dtype=torch.float64, device="cuda")
    if 2 * sum(lens) * nq * d * new > 2e13:
        return None
    for r, length in enumerate(lens):
        ids = s["table"][r, : -(-length // bs)].long()
        # keys and values of a head, token after token
        K, V = ((s[c][ids].double() * s[m][ids].double()[..., None, None] / 127).permute(1, 0, 2, 3).flatten(1, 2)[:, :length]
                for c, m in (("Kc", "Kmax"), ("Vc", "Vmax")))
        for i in range(new):
            end = length - new + i + 1
            q = s["Q"][r * new + i].double().view(nk, nq // nk, d)
            e = torch.einsum("hgd,hld->hgl", q, K[:, :end]) / math.sqrt(d)
            O[r * new + i] = torch.einsum("hgl,hld->hgd", torch.softmax(e, -1), V[:, :end]).reshape(nq, d)
    return O
