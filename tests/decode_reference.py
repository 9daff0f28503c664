"""Plain 64-bit definitions of the decode step's operators for the tests: numpy
loops written from the formulas, sharing no code with the package."""
import numpy as np

MIN_EXP = -100
QMAX = {"e4m3": 448.0, "int8": 127.0}


def plan(lens, new, table, ring, pool, page, n_tokens):
    """The documented rule, request by request."""
    R, width, n_pages = len(lens), table.shape[1], len(ring)
    table, ring = table.copy(), ring.copy()
    head, free = pool
    cu, kv = [0], []
    asked = taken = back = 0
    slots, pos, status = np.full(n_tokens, -1, np.int64), np.full(n_tokens, -1, np.int32), 0
    ring_in = ring.copy()
    for r in range(R):
        have = -(-int(lens[r]) // page)
        add = max(int(new[r]), 0)
        beg, end = cu[-1], cu[-1] + add
        cu.append(end)
        if new[r] < 0:
            for j in range(min(have, width)):
                ring[(head + free + back) % n_pages] = table[r, j]
                back += 1
            kv.append(0)
            continue
        need = -(-(int(lens[r]) + add) // page) - have
        wide = have + need > width
        asked += 0 if wide else need
        if add and (wide or (need and asked > free) or end > n_tokens):
            status = -10
            kv.append(int(lens[r]))
            continue
        if need:
            first = asked - need
            for j in range(need):
                table[r, have + j] = ring_in[(head + first + j) % n_pages]
            taken = asked
        kv.append(int(lens[r]) + add)
        for i in range(add):
            p = int(lens[r]) + i
            slots[beg + i] = int(table[r, p // page]) * page + p % page
            pos[beg + i] = p
    return dict(kv_lens=np.array(kv, np.int32), cu_q=np.minimum(cu, n_tokens).astype(np.int32), slots=slots,
                positions=pos, pool=np.array([(head + taken) % n_pages, free - taken + back], np.int32), table=table,
                ring=ring, status=status)


def round_code(x, fmt):
    """Nearest code value, ties to even."""
    if fmt == "int8":
        return np.rint(x)
    exp = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -40)))
    step = np.exp2(np.maximum(exp, -6.0) - 3)
    return np.rint(x / step) * step


def scale_of(amax, fmt):
    """2^e with the least e >= MIN_EXP such that amax <= qmax 2^e."""
    e = MIN_EXP
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scale, x, cu, slots, fmt):
    """codes [pages, heads, page, dim] and scale [pages, heads] in 64 bits, after
    x [tokens, heads, dim] (finite) went in; also whether e4m3 or int8 rounded it."""
    codes, scale = codes.astype(np.float64).copy(), scale.astype(np.float64).copy()
    page = codes.shape[2]
    for r in range(len(cu) - 1):
        own = range(cu[r], cu[r + 1])
        if len(own) == 0 or slots[cu[r]] < 0:
            continue
        for p in sorted({int(slots[t]) // page for t in own}):
            mine = [t for t in own if slots[t] // page == p]
            first = int(slots[mine[0]]) % page
            for h in range(codes.shape[1]):
                s = scale_of(max(np.abs(x[t, h]).max() for t in mine), fmt)
                if first > 0:
                    s = max(s, scale[p, h])
                    if s > scale[p, h]:
                        codes[p, h, :first] = round_code(codes[p, h, :first] * (scale[p, h] / s), fmt)
                scale[p, h] = s
                for t in mine:
                    codes[p, h, int(slots[t]) % page] = round_code(x[t, h] / s, fmt)
    return codes, scale


def attention(q, k, v, scale, limit):
    """q [rows, dim], k and v [tokens, dim] -> (o, lse, sum of p |v|, largest sum |q||k| scale)."""
    o, lse, spread, most = np.zeros(q.shape), np.full(len(q), -np.inf), np.zeros(q.shape), 0.0
    for i, n in enumerate(limit):
        if n <= 0:
            continue
        x = scale * (k[:n] @ q[i])
        m = x.max()
        p = np.exp(x - m)
        lse[i] = m + np.log(p.sum())
        p /= p.sum()
        o[i], spread[i] = p @ v[:n], p @ np.abs(v[:n])
        most = max(most, scale * float((np.abs(k[:n]) @ np.abs(q[i])).max()))
    return o, lse, spread, most


def logprobs(x, target, k):
    """One row of scaled logits x: (logprob, entropy, lse, top values, top indexes)."""
    if np.isnan(x).any() or (x == np.inf).any():
        return (np.nan if 0 <= target < len(x) else 0.0, np.nan, np.nan, np.full(k, np.nan), np.full(k, -1))
    order = sorted(range(len(x)), key=lambda j: (-x[j], j))[:k]
    has = 0 <= target < len(x)
    if (x == -np.inf).all():
        return (-np.inf if has else 0.0), 0.0, -np.inf, np.full(k, -np.inf), np.array(order)
    m = x.max()
    lse = m + np.log(np.exp(x - m).sum())
    p = np.exp(x - lse)
    live = p > 0
    return (x[target] - lse if has else 0.0, -(p[live] * (x[live] - lse)).sum(), lse, x[order] - lse, np.array(order))
