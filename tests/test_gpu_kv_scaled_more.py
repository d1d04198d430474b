"""kv.append and kv.attend over caches with scales: weights' precision, ranges
and the ways of cutting work that other tests do not reach."""
import math

import pytest
import torch

import kv_reference as ref
import kv_step_reference as step
from kv_step_reference import E4M3, F64, I8, MOST
from lossless_bf16_tensor_amd import kv
from test_gpu_kv_scaled import BF16, DEV, F16, bits, check, make, new_tokens, powers, put, step_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q", [BF16, F16])
@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("B,T,hq,H,D,S", [(1, 4, 8, 2, 128, 300), (5, 70, 32, 8, 128, 2400), (5, 70, 32, 8, 64, 2400)])
def test_weights_are_finer_than_the_output(q, cache, B, T, hq, H, D, S):
    """All weights are one number, an equal share times a scale just above the
    middle between two BF16 values, so a weight in one term of BF16 would be off by 2^-8 for all
    keys alike: 1.625 (1 + 2^-7) instead of 1.625 (1 + 2^-8), which BF16 rounds
    on to 1.6406, 9.2e-3 from 1.6314, where half its step is 3.9e-3."""
    vs = torch.full((B, -(-S // 16), H), 1 + 2.0 ** -8 + 2.0 ** -14, device=DEV)
    k, v = torch.zeros(B, S, H, D, device=DEV).to(cache), torch.full((B, S, H, D), 13.0 if cache == I8 else 1.625, device=DEV).to(cache)
    vs /= 8.0 if cache == I8 else 1.0
    n = torch.tensor([S - T - 17 * b for b in range(B)], dtype=torch.int32, device=DEV)
    out = kv.attend(torch.zeros(B, T, hq, D, dtype=q, device=DEV), k, v, n, k_scale=torch.ones_like(vs), v_scale=vs)
    want = 1.625 * (1 + 2.0 ** -8 + 2.0 ** -14)
    # a rounding of the output, 2^-16 of two terms, and a rounding of a binary32 sum for each key
    assert ((out.double() - want).abs() <= want * (ref.HALF[q] * (1 + 2.0 ** -7) + 2.0 ** -16 + S * 2.0 ** -24)).all()


@pytest.mark.parametrize("B,T,hq,H,D,S,cache,layout", [(5, 24, 96, 32, 128, 1760, I8, "shd"), (5, 70, 32, 8, 64, 2400, E4M3, "paged32")])
def test_many_rows_are_as_precise_as_few(B, T, hq, H, D, S, cache, layout):
    q, k, v, ks, vs, table = make(B, T, hq, H, D, S, BF16, cache, 16, layout, seed=B + T, dev=DEV)
    G = hq // H
    length, drafted = torch.tensor([S - T - 31 * b for b in range(B)], dtype=torch.int32), torch.full((B,), T, dtype=torch.int32)
    out = kv.attend(q, k, v, length.to(DEV), table=table, k_scale=ks, v_scale=vs)
    for b in (0, B - 1):
        args = [t[:, :, :1].cpu() for t in (k, v, ks, vs)] if table is not None else [t[b:b + 1, :, :1].cpu() for t in (k, v, ks, vs)]
        want = step_rows(q[b:b + 1, :, :G].cpu(), args, 16, length[b:b + 1], None if table is None else table[b:b + 1].cpu(), None, drafted[b:b + 1],
                         [0, T // 2, T - 1], False)
        for i, (o, ob, _, _) in want.items():
            ref.within(out[b, i, :G], o, ob, f"out {b} {i}")


@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("q", [BF16, F16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_scales_of_blocks_that_no_query_sees(cache, q, bad):
    """Drafted tokens that the tree names for nobody have no effect, whatever their
    elements and scales hold, in a cache and in pages, in few rows and in many."""
    for B, T, hq, H, D, n, layout in ((1, 40, 4, 2, 64, 48, "shd"), (2, 40, 16, 2, 128, 64, "paged16")):
        qq, k, v, ks, vs, table = make(B, T, hq, H, D, n + T, q, cache, 16, layout, seed=T)
        tree = torch.ones(T, T, dtype=torch.bool).tril()
        tree[:, 16:32] = False
        for b in range(B):
            at = (b, n // 16 + 1) if table is None else (int(table[b, n // 16 + 1]), 0)
            ks[at], vs[at] = bad, bad
        check(qq, k, v, ks, vs, table, [n] * B, tree=tree)


@pytest.mark.parametrize("layout", ["shd", "paged32"])
def test_scales_of_blocks_that_none_of_many_rows_sees(layout):
    B, T, hq, H, D, S = 5, 70, 32, 8, 128, 2400
    q, k, v, ks, vs, table = make(B, T, hq, H, D, S, F16, E4M3, 32, layout, seed=9, dev=DEV)
    G, n = hq // H, 2304                                             # of whole blocks and pages
    tree = torch.ones(T, T, dtype=torch.bool).tril()
    tree[:, 32:64] = False
    for b in range(B):
        at = (b, n // 32 + 1) if table is None else (int(table[b, n // 32 + 1]), 0)
        ks[at], vs[at] = math.nan, math.inf
    length, drafted = torch.full((B,), n, dtype=torch.int32), torch.full((B,), T, dtype=torch.int32)
    lse = torch.empty(B, T, hq, device=DEV)
    out = kv.attend(q, k, v, length.to(DEV), table=table, tree=tree.to(DEV), lse=lse, k_scale=ks, v_scale=vs)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    args = [t[:, :, :1].cpu() for t in (k, v, ks, vs)] if table is not None else [t[:1, :, :1].cpu() for t in (k, v, ks, vs)]
    want = step_rows(q[:1, :, :G].cpu(), args, 32, length[:1], None if table is None else table[:1].cpu(), tree[None], drafted[:1], [0, 31, 40, T - 1], False)
    for i, (o, ob, l, lb) in want.items():
        ref.within(out[0, i, :G], o, ob, f"out {i}")
        ref.within(lse[0, i, :G], l, lb, f"lse {i}")


@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("power", [80, -80])
@pytest.mark.parametrize("B,T,hq,H,D,S", [(1, 1, 1, 1, 8, 1 << 22), (1, 4, 8, 2, 64, 1 << 18), (5, 70, 32, 8, 128, 2400)])
def test_scales_at_the_ends_of_their_range(cache, power, B, T, hq, H, D, S):
    """The largest values. First under weights that grow by just less than what has
    the maximum raised, so that sums are of weights of 2^7.9; then all but one
    under weights of 2^-20."""
    k, v = torch.zeros(B, S, H, D, device=DEV).to(cache), torch.full((B, S, H, D), MOST[cache], device=DEV).to(cache)
    ks, vs = torch.ones(B, -(-S // 16), H, device=DEV), torch.full((B, -(-S // 16), H), 2.0 ** power, device=DEV)
    q = torch.zeros(B, T, hq, D, dtype=BF16, device=DEV)
    q[..., 0] = 1.0
    n = torch.full((B,), S - T, dtype=torch.int32, device=DEV)
    k.view(torch.uint8)[:, S // 32:, :, 0] = torch.full((1,), 64.0, device=DEV).to(cache).view(torch.uint8)
    ks.fill_(7.9 * math.log(2) * math.sqrt(D) / 64)
    want = MOST[cache] * 2.0 ** power
    out = kv.attend(q, k, v, n, k_scale=ks, v_scale=vs).double()
    # the output's rounding; sums of each wave, and of the waves, of 2^12 roundings at most
    assert ((out / want - 1).abs() <= 2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -11).all()
    k.view(torch.uint8).zero_()
    k.view(torch.uint8)[:, 5, :, 0] = torch.full((1,), 64.0, device=DEV).to(cache).view(torch.uint8)
    v.view(torch.uint8)[:, 5] = 0
    ks.fill_(20 * math.log(2) * math.sqrt(D) / 64)
    out = kv.attend(q, k, v, n, k_scale=ks, v_scale=vs).double()
    for i in range(T):
        others = (S - T + i) * 2.0 ** -20
        assert ((out[:, i] / (want * others / (1 + others)) - 1).abs() <= 2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -11).all()


@pytest.mark.parametrize("cache", [I8, E4M3])
def test_scales_of_the_farthest_strides(cache):
    """Scales whose last one is element 2^30 - 1 of their memory: the same output and cache as with scales side by side."""
    H, D, page, block = 2, 64, 32, 16
    first = (2 ** 30 - 1 - 64 - 7) // 2
    assert 2 * first + 64 + 7 == 2 ** 30 - 1
    q, k, v, ks, vs, _ = make(1, 3, 4, H, D, 70, BF16, cache, block, "paged32", seed=3, dev=DEV)
    k, v, ks, vs = k[:3].clone(), v[:3].clone(), ks[:3].contiguous(), vs[:3].contiguous()
    table, n = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV), torch.tensor([70], dtype=torch.int32, device=DEV)
    far = [torch.zeros(2 ** 30, device=DEV).as_strided((3, 2, H), (first, 64, 7)) for _ in "kv"]
    for a, b in zip(far, (ks, vs)):
        a.copy_(b)
    new = (torch.randn(1, 3, H, D, device=DEV) * 40).to(BF16)
    got = []
    for s in ((ks, vs), far):
        kk, vv = k.clone(), v.clone()
        kv.append(None, new, new, kk, vv, n, table=table, k_scale=s[0], v_scale=s[1])
        got.append([x.contiguous().view(torch.uint8) for x in (kv.attend(q, kk, vv, n, table=table, k_scale=s[0], v_scale=s[1]), kk, vv, *s)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


# long ragged batches of few rows, where each workgroup takes its share of all sequences
WALKS = [(32, 1, 16, 8, 128, 8200, BF16, E4M3, 16, "paged64", False), (20, 4, 32, 8, 128, 13200, BF16, I8, 32, "paged32", True),
         (64, 3, 32, 16, 120, 4200, F16, I8, 64, "hsd", True), (7, 16, 32, 32, 72, 10000, F16, E4M3, 16, "paged16", False),
         (100, 2, 32, 16, 128, 1400, BF16, I8, 128, "paged128", True), (16, 8, 16, 8, 128, 16400, F16, E4M3, 32, "shd", True)]


@pytest.mark.parametrize("B,T,hq,H,D,S,qt,cache,block,layout,with_tree", WALKS)
def test_shares_of_all_sequences(B, T, hq, H, D, S, qt, cache, block, layout, with_tree):
    """Ragged and empty sequences, fewer drafted tokens than given, absent pages, a
    value that is NaN in a drafted token of a sequence that many workgroups share."""
    q, k, v, ks, vs, table = make(B, T, hq, H, D, S, qt, cache, block, layout, seed=B + T, dev=DEV)
    g = torch.Generator().manual_seed(B)
    G = hq // H
    length = (torch.rand(B, generator=g) ** 3 * (S - T)).to(torch.int32)
    drafted = torch.randint(1, T + 1, (B,), generator=g).to(torch.int32)
    length[0], drafted[0] = S - T, T                  # the longest, in many parts
    length[1], length[3], drafted[3], drafted[4] = 0, 0, 0, 0
    length[B - 1], drafted[B - 1] = S - T - 1, T
    tree = None
    if with_tree:
        tree = torch.rand(B, T, T, generator=g) < 0.5
        tree[:, T - 1] = False
    if table is not None:
        page = k.shape[1]
        table[0, 3] = -1
        table[0, (S - T) // page - 1] = k.shape[0] + 7
        table[B - 1, 0] = -1
    if cache == E4M3:
        n = S - T                                      # the first drafted token of sequence 0
        at = (0, n) if table is None else (int(table[0, n // page]), n % page)
        bits(v)[at][:, 5] = 0x7f
        if with_tree:
            tree[0, :, 0] = torch.arange(T) % 2 == 0
    kk, vv, kks, vvs = (put(t.cpu(), layout) for t in (k, v, ks, vs))
    got = []
    for _ in range(2):
        lse, w = torch.empty(B, T, hq, device=DEV), torch.zeros(B, H, S if table is None else table.shape[1] * page, device=DEV)
        out = kv.attend(q, kk, vv, length.to(DEV), table=table, tree=put(tree), drafted=drafted.to(DEV), lse=lse, score=w, k_scale=kks, v_scale=vvs)
        got.append((out, lse, w))
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(*got))
    for b in sorted({0, 1, 2, 3, 4, 5, B // 2, B - 2, B - 1}):
        for h in sorted({0, H - 1}):
            args = [t[:, :, h:h + 1].cpu() for t in (k, v, ks, vs)] if table is not None else [t[b:b + 1, :, h:h + 1].cpu() for t in (k, v, ks, vs)]
            want = step_rows(q[b:b + 1, :, h * G:h * G + G].cpu(), args, block, length[b:b + 1], None if table is None else table[b:b + 1].cpu(),
                             None if tree is None else tree[b:b + 1], drafted[b:b + 1], sorted({0, 1 % T, T - 1}), False)
            for i, (o, ob, l, lb) in want.items():
                ref.within(out[b, i, h * G:h * G + G], o, ob, f"out {b} {i} {h}")
                ref.within(lse[b, i, h * G:h * G + G], l, lb, f"lse {b} {i} {h}")
    assert torch.isnan(out[0, 0, :, 5]).all() == (cache == E4M3)
    seeing = torch.isfinite(lse).sum((1, 2)).double().cpu()
    assert ((w.double().sum((1, 2)).cpu() - seeing).abs() <= seeing * 2.0 ** -10).all()


@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("layout", ["shd", "paged32"])
def test_accepted_tokens_of_a_tree_are_appended_again(cache, layout):
    """Over caches with scales the accepted nodes' keys and values go in once more, as
    a chain. Earlier tokens of a block keep the scale that a rejected one raised."""
    B, T, H, D, S, block = 2, 12, 2, 64, 96, 16
    _, k, v, ks, vs, table = make(B, 1, H, H, D, S, BF16, cache, block, layout, seed=4)
    ks, vs = powers(ks), powers(vs)
    nk, nv = new_tokens(B, T, H, D, BF16, 5)
    nk[:, 5], nv[:, 6] = nk[:, 5] * 64, nv[:, 6] * 64                   # rejected, and far larger than the others
    n = torch.tensor([40, 63], dtype=torch.int32)
    path, count = torch.tensor([[0, 3, 7, 8], [0, 1, 11, 11]]), torch.tensor([4, 3], dtype=torch.int32)
    dk, dv, dks, dvs = (t.to(DEV) for t in (k, v, ks, vs))
    way = [torch.stack([x[b, path[b]] for b in range(B)]) for x in (nk, nv)]
    kv.append(None, nk.to(DEV), nv.to(DEV), dk, dv, n.to(DEV), table=put(table), k_scale=dks, v_scale=dvs)
    kv.append(None, way[0].to(DEV), way[1].to(DEV), dk, dv, n.to(DEV), table=put(table), drafted=count.to(DEV), k_scale=dks, v_scale=dvs)
    for got, s, c, cs, x, y in ((dk, dks, k, ks, nk, way[0]), (dv, dvs, v, vs, nv, way[1])):
        once, s1, _ = step.append8(c, cs, x.to(F64), n, None, table, block)
        want, s2, _ = step.append8(once.to(cache), s1.float(), y.to(F64), n, count, table, block)
        assert torch.equal(s.cpu().to(F64), s2) and (s2 > cs.to(F64) * 8).any()
        for b in range(B):
            for t in range(int(n[b] + count[b])):
                at = step.place(c, table, b, t)
                assert torch.equal(got[at].cpu().to(F64), want[at]), (b, t)
