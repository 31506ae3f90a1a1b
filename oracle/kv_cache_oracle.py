"""Float64 oracle of the key/value cache in 8 bits (plain loops; test infrastructure only)."""
import numpy as np


def plan(add, lens, table, free, taken, bs, rows):
    """(status, lens, taken, cu, pos, slots, table) after a step; a step that does not fit changes nothing."""
    n, width = table.shape
    table, status = table.copy(), 0
    cu, first, used = [0], [], int(taken)
    if taken < 0:
        status |= 1
    for r in range(n):
        a, old = int(add[r]), int(lens[r])
        if a < 0 or old < 0:
            status |= 8
            a, old = max(a, 0), max(old, 0)
        have, need = -(-old // bs), -(-(old + a) // bs)
        if need > width:
            status |= 2
        first.append(used)
        used += need - have
        cu.append(cu[-1] + a)
    if used > len(free):
        status |= 1
    if cu[-1] > rows:
        status |= 4
    pos, slots = np.zeros(rows, np.int32), np.full(rows, -1, np.int32)
    if status:
        return status, lens.copy(), int(taken), np.zeros(n + 1, np.int32), pos, slots, table
    for r in range(n):
        old = int(lens[r])
        have, need = -(-old // bs), -(-(old + int(add[r])) // bs)
        for b in range(have, need):
            table[r, b] = free[first[r] + b - have]
        for i in range(int(add[r])):
            p = old + i
            s = int(table[r, p // bs]) * bs + p % bs
            pos[cu[r] + i], slots[cu[r] + i] = p, s if -(2**31) <= s < 2**31 else -1
    return 0, (lens + add).astype(np.int32), used, np.array(cu, np.int32), pos, slots, table


def write(x, slots, codes, most):
    """The cache after rows x [tokens, nk, d] (float64) went to their slots: codes [blocks, nk, bs, d] int8, most [blocks, nk]."""
    codes, most = codes.copy(), most.astype(np.float64)
    blocks, nk, bs, d = codes.shape
    runs = []
    for t, s in enumerate(slots):
        if not 0 <= s < blocks * bs:
            continue
        if runs and t > 0 and runs[-1][-1][0] == t - 1 and slots[t - 1] == s - 1 and s % bs:
            runs[-1].append((t, s))
        else:
            runs.append([(t, s)])
    for run in runs:
        block, off = divmod(int(run[0][1]), bs)
        rows = x[[t for t, _ in run]]  # [run, nk, d]
        for h in range(nk):
            new = rows[:, h]
            old = most[block, h] if off else 0.0
            top = max(old, float(np.abs(new).max())) if np.isfinite(new).all() and np.isfinite(old) else np.nan
            held = codes[block, h, :off].astype(np.float64)
            if np.isfinite(top) and off and top != old:
                codes[block, h, :off] = np.rint(held * old / top).astype(np.int8) if top > 0 else 0
            c = np.zeros_like(new)
            if np.isfinite(top) and top >= 2.0**-80:
                c = np.rint(new * 127 / top)
            codes[block, h, off : off + len(run)] = c.astype(np.int8)
            most[block, h] = top
    return codes, most


def attn(q, Kc, Vc, Kmax, Vmax, table, length, scale):
    """One request: q [m, nq, d] its last m tokens' queries.  (O, weighted mean of |v|, largest scale sum |q k| of a row),
    [m, nq, d], [m, nq, d], [m, nq]; pages outside the pool and what is behind the table are left out."""
    m, nq, d = q.shape
    blocks, nk, bs, _ = Kc.shape
    here = [(j, int(table[j // bs])) for j in range(max(0, min(length, len(table) * bs)))]
    here = [(j, b) for j, b in here if 0 <= b < blocks]
    O, A, E = np.zeros((m, nq, d)), np.zeros((m, nq, d)), np.zeros((m, nq))
    js = np.array([j for j, _ in here], dtype=np.int64)
    bl = np.array([b for _, b in here], dtype=np.int64)
    for h in range(nk):
        K = Kc[bl, h, js % bs].astype(np.float64) * (Kmax[bl, h].astype(np.float64) / 127)[:, None] if len(js) else np.zeros((0, d))
        V = Vc[bl, h, js % bs].astype(np.float64) * (Vmax[bl, h].astype(np.float64) / 127)[:, None] if len(js) else np.zeros((0, d))
        for i in range(m):
            see = js <= length - m + i
            if not see.any():
                continue
            for g in range(h * (nq // nk), (h + 1) * (nq // nk)):
                s = K[see] @ q[i, g] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                O[i, g], A[i, g] = p @ V[see], p @ np.abs(V[see])
                E[i, g] = (np.abs(K[see]) @ np.abs(q[i, g])).max() * scale
    return O, A, E
