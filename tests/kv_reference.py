"""Plain 64-bit forms of the KV-cache operators, one sequence and head at a
time on the CPU, and the bounds that their kernels' results must keep."""
import math

import torch

F64 = torch.float64
# half a step of a type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e5m2: 2.0 ** -3, torch.float32: 2.0 ** -24}
# half the smallest subnormal step
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float8_e5m2: 2.0 ** -17}


def turned(x, pos, freq, amplitude=1.0, interleaved=False, inverse=False):
    """x [B, T, H, D] in 64 bits, turned; pos [B, T]."""
    y = x.to(F64).clone()
    half = freq.numel()
    angle = 2.0 * math.pi * torch.remainder(pos.to(F64)[..., None] * freq, 1.0)
    cos, sin = (f(angle)[:, :, None, :] * amplitude for f in (torch.cos, torch.sin))
    if inverse:
        sin = -sin
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * cos - w * sin
    y[..., b] = w * cos + u * sin
    return y


def rope_bound(x, want, freq, amplitude, dtype):
    """One rounding to the type; in binary32 two products and a sum on cos and
    sin that are off by 2^-22 (the fraction of a turn rounded to binary32, times
    2 pi, and the functions' own error)."""
    size = x.to(F64).abs().amax(-1, keepdim=True)
    return want.abs() * HALF[dtype] * (1 + 2.0 ** -8) + TINY[dtype] + abs(amplitude) * size * 2.0 ** -20


def rows_of(cache, table, b, n):
    """The first n tokens of sequence b, [n, heads, dim] in 64 bits, and which of them are there."""
    if table is None:
        return cache[b, :n].to(F64), torch.ones(n, dtype=torch.bool)
    page = cache.shape[1]
    p = table[b, torch.arange(n) // page].long()
    there = (p >= 0) & (p < cache.shape[0])
    rows = cache.to(F64)[torch.where(there, p, 0), torch.arange(n) % page]
    return rows, there


def attend(q, k, v, length, *, table=None, tree=None, drafted=None, scale=None):
    """{out, lse, weight} and the bounds {out_bound, lse_bound, weight_bound}; weight is [B, H, tokens]."""
    B, T, hq, D = q.shape
    H = k.shape[2]
    G = hq // H
    cap = k.shape[1] if table is None else table.shape[1] * k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, bound = torch.zeros(B, T, hq, D, dtype=F64), torch.zeros(B, T, hq, D, dtype=F64)
    lse, lse_bound = torch.full((B, T, hq), -math.inf, dtype=F64), torch.zeros(B, T, hq, dtype=F64)
    weight, weight_bound = torch.zeros(B, H, cap, dtype=F64), torch.zeros(B, H, cap, dtype=F64)
    for b in range(B):
        n = max(0, min(int(length[b]), cap))
        t = T if drafted is None else max(0, min(int(drafted[b]), T))
        end = min(n + t, cap) if t else 0
        kk, there = rows_of(k, table, b, end)
        vv, _ = rows_of(v, table, b, end)
        for i in range(t):
            see = there.clone()
            for j in range(max(0, end - n)):
                if tree is not None:
                    see[n + j] &= bool(tree[b, i, j] if tree.dim() == 3 else tree[i, j])
                else:
                    see[n + j] &= j <= i
            at = see.nonzero()[:, 0]
            if not at.numel():
                continue
            for a in range(hq):
                x = q[b, i, a].to(F64)
                kh, vh = kk[at, a // G], vv[at, a // G]
                s = scale * (kh @ x)
                top = s.max()
                if top == -math.inf:
                    continue
                p = torch.exp(s - top)
                total = p.sum()
                lse[b, i, a] = top + total.log()
                p = p / total
                out[b, i, a] = p @ vh
                weight[b, a // G, at] += p
                # a score is a binary32 sum of D exact products, then a few
                # roundings of it, of the maximum and of 2^x
                size = float((scale * (kh.abs() @ x.abs())).max()) if math.isfinite(float(s.abs().max())) else 0.0
                ds = (D + 16) * 2.0 ** -23 * size + 2.0 ** -21 * (1.0 + size)
                sums = at.numel() * 2.0 ** -24
                narrow = torch.float16 if k.dtype != torch.bfloat16 else torch.bfloat16
                spread = p @ vh.abs()
                bound[b, i, a] = ((HALF[narrow] * (1 + 2.0 ** -7) + 2 * ds + sums) * spread
                                  + TINY[narrow] * vh.abs().sum(0) / total * 2
                                  + HALF[q.dtype] * (1 + 2.0 ** -7) * out[b, i, a].abs() + TINY[q.dtype])
                lse_bound[b, i, a] = 2 * ds + sums + 2.0 ** -22 * float(lse[b, i, a].abs())
                weight_bound[b, a // G, at] += p * (4 * ds + sums + 2.0 ** -22 * (1 + float(lse[b, i, a].abs()))) + 2.0 ** -120
        weight_bound[b] += weight[b] * (T * G) * 2.0 ** -24
    return dict(out=out, lse=lse, weight=weight, out_bound=bound, lse_bound=lse_bound, weight_bound=weight_bound)


def evict(score, length, keep, sink, recent, cap):
    """[B][H] lists of kept tokens."""
    kept = []
    for b in range(score.shape[0]):
        n = max(0, min(int(length[b]), cap))
        per = []
        for h in range(score.shape[1]):
            def worth(i):
                s = float(score[b, h, i])
                return (0 if i < sink or i >= n - recent else 1, -s if s == s else math.inf, i)
            per.append(sorted(sorted(range(n), key=worth)[:keep]))
        kept.append(per)
    return kept


def within(got, want, bound, what=""):
    """Every element within its bound; NaN where NaN is wanted, infinities equal."""
    got, want = got.detach().cpu().to(F64), want.to(F64)
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), f"{what}: infinities differ"
    off = (got - want).abs()[~odd] - bound.expand_as(want)[~odd]
    if off.numel() and float(off.max()) > 0:
        worst = int(off.argmax())
        raise AssertionError(f"{what}: {got[~odd][worst]} for {want[~odd][worst]}, bound {bound.expand_as(want)[~odd][worst]}, "
                             f"{int((off > 0).sum())} of {off.numel()} outside")
