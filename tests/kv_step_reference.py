"""Plain 64-bit forms of the operators of drafted tokens and of 8-bit caches
with scales, one sequence, head or page at a time on the CPU."""
import math

import torch

import kv_reference as ref

F64 = torch.float64
E4M3, I8 = torch.float8_e4m3fn, torch.int8
MOST = {E4M3: 448.0, I8: 127.0}


def place(cache, table, b, t):
    """(first, second) index of token t of sequence b, or None outside the cache or in an absent page."""
    if table is None:
        return (b, t) if 0 <= t < cache.shape[1] else None
    page = cache.shape[1]
    if not 0 <= t < table.shape[1] * page:
        return None
    p = int(table[b, t // page])
    return (p, t % page) if 0 <= p < cache.shape[0] else None


def rounded(y, dtype):
    """float64 to the nearest of the type's values, ties to even; beyond them the largest, NaN to NaN or 0."""
    if dtype == I8:
        return torch.nan_to_num(torch.round(y).clamp(-127, 127), nan=0.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6, max=448.0))) - 3.0)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def scale_for(a, most):
    e = -60
    while a > 2.0 ** e * most:
        e += 1
    return 2.0 ** e


def append8(cache, scale, x, length, drafted, table, block):
    """A cache [.., tokens, heads, dim] and its scales after new tokens x [B, T, H, D] (float64); returns them in float64, and where was written."""
    most = MOST[cache.dtype]
    got, s = cache.to(F64), scale.to(F64)
    written = torch.zeros(cache.shape[:2], dtype=torch.bool)
    B, T = x.shape[:2]
    for b in range(B):
        n = int(length[b])
        blocks = {}
        for t in range(T if drafted is None else max(0, min(T, int(drafted[b])))):
            at = place(cache, table, b, n + t)
            if at is not None:
                blocks.setdefault((at[0], at[1] // block), []).append((t, at))
        for (first, blk), new in blocks.items():
            start = n + new[0][0] - new[0][1][1] % block           # the block's first token
            earlier = [place(cache, table, b, t) for t in range(max(start, 0), max(min(n, start + block), 0))]
            for h in range(x.shape[2]):
                rows = torch.stack([x[b, t, h] for t, _ in new])
                fine = rows.abs()[torch.isfinite(rows)]
                a = float(fine.max()) if fine.numel() else 0.0
                old = float(s[first, blk, h])
                now = old if earlier and a <= old * most else scale_for(a, most)
                for at in earlier:
                    if now != old:
                        got[at][h] = rounded(got[at][h] * (old / now), cache.dtype)
                for (t, at), row in zip(new, rows):
                    got[at][h] = rounded(row / now, cache.dtype)
                    written[at] = True
                for at in earlier:
                    written[at] = True
                s[first, blk, h] = now
    return got, s, written


def whole(cache, scale, block):
    """What the elements of a cache stand for, in float64."""
    return cache.to(F64) * scale.to(F64).repeat_interleave(block, 1)[:, :cache.shape[1], :, None]


def attend8(q, k, v, ks, vs, block, length, coarse=False, **kw):
    """kv_reference.attend over what the elements stand for. coarse: weights in
    one term of BF16, off by half a step of it, not in two, off by 2^-16, which
    the bound of FP16 weights covers."""
    k, v = whole(k, ks, block), whole(v, vs, block)
    want = ref.attend(q, k, v, length, **kw)
    if coarse:
        spread = ref.attend(q, k, v.abs(), length, **kw)["out"]
        want["out_bound"] = want["out_bound"] + 2.0 ** -8 * (1 + 2.0 ** -7) * spread
    return want


def verify(tokens, target, uniform, draft=None, parent=None, drafted=None):
    """Per sequence (path, count, token), in Python's floats."""
    B, T, V = target.shape
    found = []
    for b in range(B):
        nd = T if drafted is None else max(0, min(T, int(drafted[b])))
        if not nd:
            found.append(([], 0, -1))
            continue
        clean = lambda t: torch.where(torch.isfinite(t) & (t > 0), t, torch.zeros_like(t)).double()  # noqa: E731
        at, path = 0, [0]
        while True:
            left, mass, gone, nxt = clean(target[b, at]), 1.0, set(), None
            q = clean(draft[b, at]) if draft is not None else None
            for i in range(at + 1, nd):
                up = i - 1 if parent is None else int(parent[b, i] if parent.dim() == 2 else parent[i])
                x = int(tokens[b, i])
                if up != at or not 0 <= x < V:
                    continue
                px, qx = float(left[x]), 1.0 if q is None else float(q[x])
                if px > 0 and x not in gone and float(uniform[b, i]) * qx * mass < px:
                    nxt = i
                    break
                if q is not None:
                    left = (left - mass * q).clamp(min=0.0)
                    mass = float(left.sum())
                elif x not in gone:
                    mass -= px
                    left[x] = 0.0
                    gone.add(x)
            if nxt is None:
                break
            at = nxt
            path.append(at)
        if not bool((left > 0).any()):
            left = clean(target[b, at])
        sums = left.cumsum(0)
        there = (left > 0).nonzero()[:, 0]
        past = (sums > float(uniform[b, 0]) * float(sums[-1])).nonzero()[:, 0]
        token = -1 if not there.numel() else min(int(past[0]) if past.numel() else V, int(there[-1]))
        found.append((path, len(path), token))
    return found


def fork(table, length, parent, pages, page, room=0, held=None):
    """(table, length, moves, left) as lists."""
    rows, entries = table.shape
    there = lambda x: 0 <= x < pages  # noqa: E731
    seqs = []
    for p in parent.tolist():
        live = 0 <= p < rows
        seqs.append((table[p].tolist() if live else [], max(0, min(int(length[p]), entries * page)) if live else 0, live))
    used = {i for i in range(pages) if held is not None and bool(held[i])}
    for row, n, _ in seqs:
        used |= {x for x in row[:n // page] if there(x)}
    lasts, copies = set(), []
    for row, n, _ in seqs:
        x = row[n // page] if n % page else -1
        copies.append(n % page > 0 and there(x) and (x in used or x in lasts))
        if n % page and there(x) and x not in used:
            lasts.add(x)
    taken = used | lasts
    free = [i for i in range(pages) if i not in taken]
    out, moves, given = [], [], 0
    for (row, n, live), copy in zip(seqs, copies):
        new = [x if there(x) else -1 for x in row[:n // page]]
        if n % page and not copy:
            new.append(row[n // page] if there(row[n // page]) else -1)
        end = min(-(-(n + room) // page), entries) if live else 0
        move = (-1, -1)
        while len(new) < end:
            got = free[given] if given < len(free) else -1
            given += 1
            if copy and len(new) == n // page and got >= 0:
                move = (row[n // page], got)
            new.append(got)
        out.append(new + [-1] * (entries - len(new)))
        moves.append(list(move))
    return out, [n for _, n, _ in seqs], moves, len(free) - given


def compact(table, length, pages, page, held=None):
    """(table, moves, used) as lists."""
    entries = table.shape[1]
    rows = [[x if 0 <= x < pages else -1 for x in row[:-(-max(0, min(int(n), entries * page)) // page)]] for row, n in zip(table.tolist(), length)]
    fixed = {i for i in range(pages) if held is not None and bool(held[i])}
    mine = {x for row in rows for x in row if x >= 0}
    used = mine | fixed
    n = len(used)
    to = dict(zip(sorted(x for x in mine - fixed if x >= n), (i for i in range(n) if i not in used)))
    out = [[to.get(x, x) for x in row] + [-1] * (entries - len(row)) for row in rows]
    return out, [list(m) for m in sorted(to.items())], n


assert math.isclose(scale_for(127.0, 127.0), 1.0)
