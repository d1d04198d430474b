"""kv.append and kv.attend over caches in 8 bits with scales, against their
64-bit forms."""
import math

import pytest
import torch

import kv_reference as ref
import kv_step_reference as step
from kv_step_reference import E4M3, F64, I8, MOST
from lossless_bf16_tensor_amd import kv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16 = torch.bfloat16, torch.float16


def bits(t):
    return t.view(torch.uint8)


def filled(first, second, H, D, dtype, block, g, spread=0.5, layout="shd"):
    """A cache's elements of every value but NaN and its scales, no powers of two, on the device of g."""
    dev = g.device
    if dtype == I8:
        t = torch.randint(-128, 128, (first, second, H, D), generator=g, device=dev).to(I8)
    else:
        t = (torch.randn(first, second, H, D, generator=g, device=dev) * 100).clamp(-448, 448).to(E4M3)
    s = torch.exp(spread * torch.randn(first, -(-second // block), H, generator=g, device=dev)) / MOST[dtype] * 2
    return t, s


def make(B, T, hq, H, D, S, q=BF16, cache=I8, block=16, layout="shd", seed=0, dev="cpu", kscale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    qq = torch.randn(B, T, hq, D, generator=g, device=dev).to(q)
    table = None
    first, second = B, S
    if layout.startswith("paged"):
        second = int(layout[5:])
        per = -(-S // second)
        first = B * per + 2
        table = torch.randperm(first, generator=g, device=dev)[:B * per].view(B, per).to(torch.int32)
    (k, ks), (v, vs) = (filled(first, second, H, D, cache, block, g) for _ in "kv")
    return qq, k, v, ks * kscale, vs, table


def put(t, layout="shd"):
    if t is None:
        return None
    if layout == "hsd":
        if t.dim() == 4:
            return bits(t).transpose(1, 2).contiguous().to(DEV).transpose(1, 2).view(t.dtype)
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    return t.to(DEV)


def check(q, k, v, ks, vs, table, length, block=16, tree=None, drafted=None, layout="shd", score=True, coarse=False, **kw):
    B, T, hq, D = q.shape
    cap = k.shape[1] if table is None else table.shape[1] * k.shape[1]
    length = torch.tensor(length, dtype=torch.int32)
    drafted = None if drafted is None else torch.tensor(drafted, dtype=torch.int32)
    want = step.attend8(q, k, v, ks, vs, block, length, coarse, table=table, tree=tree, drafted=drafted)
    lse = torch.full((B, T, hq), 7.0, device=DEV)
    w = torch.full((B, k.shape[2], cap), 0.25, device=DEV) if score else None
    out = kv.attend(put(q), put(k, layout), put(v, layout), length.to(DEV), table=put(table), tree=put(tree), drafted=put(drafted), score=w, lse=lse,
                    k_scale=put(ks, layout), v_scale=put(vs, layout), **kw)
    ref.within(out, want["out"], want["out_bound"], "out")
    ref.within(lse, want["lse"], want["lse_bound"], "lse")
    if score:
        ref.within(w, want["weight"] + 0.25, want["weight_bound"] + 2.0 ** -24 * (want["weight"] + 0.25), "score")
    return out, lse, w


# ----------------------------------------------------------------- attend --
@pytest.mark.parametrize("n", [0, 1, 14, 15, 16, 31, 32, 33, 64, 100, 257, 1000, 2500])
@pytest.mark.parametrize("cache", [I8, E4M3])
def test_one_token(n, cache):
    q, k, v, ks, vs, _ = make(1, 1, 8, 2, 128, n + 1, cache=cache, seed=n)
    check(q, k, v, ks, vs, None, [n])


@pytest.mark.parametrize("q,cache", [(BF16, I8), (F16, I8), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("D", [8, 16, 64, 72, 128, 200, 256])
def test_types_and_head_dims(q, cache, D):
    for T, hq, H in ((1, 6, 2), (7, 8, 2), (21, 10, 5)):
        a, k, v, ks, vs, _ = make(2, T, hq, H, D, 150 + T, q, cache, 32, seed=D + T)
        check(a, k, v, ks, vs, None, [150, 61], 32, drafted=[T, T])


@pytest.mark.parametrize("T,hq,H", [(1, 1, 1), (2, 7, 1), (17, 1, 1), (5, 16, 2), (9, 14, 2), (33, 8, 2), (65, 4, 1), (130, 3, 1)])
def test_row_counts(T, hq, H):
    q, k, v, ks, vs, _ = make(1, T, hq, H, 64, 200 + T, cache=E4M3, block=64, seed=T)
    check(q, k, v, ks, vs, None, [200], 64)
    q, k, v, ks, vs, _ = make(1, T, hq, H, 256, 40 + T, seed=T + 1)
    check(q, k, v, ks, vs, None, [37])


@pytest.mark.parametrize("layout", ["shd", "hsd", "paged16", "paged32", "paged128"])
@pytest.mark.parametrize("block", [16, 32, 128])
@pytest.mark.parametrize("cache", [I8, E4M3])
def test_layouts_blocks_and_ragged_lengths(layout, block, cache):
    if layout.startswith("paged"):
        block = min(block, int(layout[5:]))
    q, k, v, ks, vs, table = make(5, 4, 8, 4, 128, 300, BF16, cache, block, layout, seed=3)
    check(q, k, v, ks, vs, table, [296, 0, 1, 100, 250], block, drafted=[4, 4, 0, 3, 1], layout=layout)


@pytest.mark.parametrize("T", [1, 13, 33, 70])
@pytest.mark.parametrize("n", [0, 5, 64])
def test_trees(T, n):
    """Any mask, rows that see no drafted token and (n = 0) nothing at all among them."""
    q, k, v, ks, vs, _ = make(2, T, 4, 2, 128, n + T, cache=E4M3, seed=T + n)
    tree = torch.rand(2, T, T, generator=torch.Generator().manual_seed(T)) < 0.3
    tree[:, T // 2] = False
    out, lse, _ = check(q, k, v, ks, vs, None, [n, n], tree=tree, drafted=[T, max(0, T - 2)])
    if n == 0:
        assert not out[:, T // 2].any() and torch.isinf(lse[:, T // 2]).all()


def test_absent_pages_and_lengths_outside():
    q, k, v, ks, vs, table = make(4, 3, 4, 2, 64, 200, cache=E4M3, block=32, layout="paged32", seed=8)
    table[0, 2] = -1
    table[1, 0] = k.shape[0]
    table[2] = -7
    ks[0], vs[0] = math.nan, math.inf                  # page 0 may lie behind the ends
    table[table == 0] = -1
    check(q, k, v, ks, vs, table, [190, 150, 64, 10 ** 6], 32)
    check(q, k, v, ks, vs, table, [-5, 0, 224, 199], 32, drafted=[3, 9, -1, 2])


@pytest.mark.parametrize("T,hq", [(6, 4), (20, 8), (40, 8)])
def test_masked_values_have_no_effect(T, hq):
    """NaN in keys and values that some queries do not see, and in elements and scales behind the last token."""
    n = 45
    q, k, v, ks, vs, _ = make(1, T, hq, 2, 64, n + T + 60, cache=E4M3, seed=T)
    tree = torch.eye(T, dtype=torch.bool)
    tree[:, 0] = True
    bits(k)[:, n + 2] = 0x7f
    bits(v)[:, n + 3] = 0xff
    bits(v)[:, n + 4, :, 5] = 0x7f
    for t in (k, v):
        bits(t)[:, n + T:] = 0x7f
    for s in (ks, vs):
        s[:, -(-(n + T) // 16):] = math.nan
    out, lse, _ = check(q, k, v, ks, vs, None, [n], tree=tree)
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2]).all() and torch.isnan(out[0, 3]).all()
    assert torch.isnan(out[0, 4, :, 5]).all() and not torch.isnan(out[0, 4, :, 6]).any() and not torch.isnan(out[0, 5]).any()


@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("q", [BF16, F16])
def test_scales_far_apart(cache, q):
    """Values of 2^-40 beside ones of 2^20 that hardly weigh anything: a weight
    times a scale keeps binary32's range, so that neither is lost nor overflows."""
    a, k, v, ks, vs, _ = make(1, 3, 8, 2, 64, 131, q, cache, seed=4)
    k, ks = torch.zeros_like(bits(k)).view(k.dtype), torch.ones_like(ks)
    n = torch.tensor([128], dtype=torch.int32)
    bits(k)[:, :64, :, 0] = bits(torch.full((1,), 20.0).to(cache))
    for first, second, size in ((2.0 ** -40, 2.0 ** 20, 64.0), (2.0 ** 40, 2.0 ** -60, 4.0)):
        a[..., 0] = size                    # scores of 160, so that the others' weight is below 2^-224, or of 10
        vs[:, :4], vs[:, 4:] = first / MOST[cache], second / MOST[cache]
        if q == F16:                        # an output that FP16 holds
            vs *= 1.0 / first
        got = kv.attend(put(a), put(k), put(v), n.to(DEV), k_scale=put(ks), v_scale=put(vs)).cpu().to(F64)
        want = step.attend8(a, k, v, ks, vs, 16, n)["out"]
        spread = step.attend8(a, k, torch.ones_like(v), ks, vs * MOST[cache], 16, n)["out"]
        assert ((got - want).abs() <= want.abs() * ref.HALF[q] * 1.01 + spread * 2.0 ** -14 + ref.TINY[q]).all()


def test_scales_stay_in_order():
    """Scales of any strides, a view of a larger tensor."""
    q, k, v, ks, vs, _ = make(2, 2, 8, 4, 64, 100, cache=I8, seed=2)
    n = torch.tensor([98, 40], dtype=torch.int32, device=DEV)
    want = kv.attend(put(q), put(k), put(v), n, k_scale=put(ks), v_scale=put(vs))
    wide = torch.full((2, 4, 7, 3), math.nan, device=DEV)
    wide[..., 1] = ks.transpose(1, 2).to(DEV)
    got = kv.attend(put(q), put(k), put(v), n, k_scale=wide[..., 1].transpose(1, 2), v_scale=put(vs, "hsd"))
    assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB whose last pages are used, and scales behind 2^31 elements of their strides."""
    H, D, page, pages = 8, 256, 1024, 2400
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randint(-127, 128, (pages, page, H, D), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (pages, page, H, D), generator=g, device=DEV, dtype=torch.int8)
    ks = torch.rand(pages, page // 16, H, generator=g, device=DEV) * 0.02
    vs = torch.rand(pages, page // 16, H, generator=g, device=DEV) * 0.02
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32)
    q = torch.randn(1, 2, 8, D, generator=g, device=DEV).to(BF16)
    out = kv.attend(q, k, v, torch.tensor([2500], dtype=torch.int32, device=DEV), table=table.to(DEV), k_scale=ks, v_scale=vs)
    at = table[0].long().to(DEV)
    few = torch.arange(3, dtype=torch.int32)[None]
    want = step.attend8(q.cpu(), k[at].cpu(), v[at].cpu(), ks[at].cpu(), vs[at].cpu(), 16, torch.tensor([2500]), table=few)
    ref.within(out, want["out"], want["out_bound"], "out")


SHARED = [(5, 24, 96, 32, 128, 1760, BF16, I8, 16, "shd"), (5, 70, 32, 8, 128, 2400, BF16, E4M3, 16, "paged16"), (5, 70, 32, 8, 64, 2400, F16, I8, 32, "paged32"),
          (5, 24, 96, 32, 80, 1760, F16, E4M3, 64, "hsd"), (5, 33, 64, 32, 48, 1800, F16, I8, 128, "hsd"), (1, 64, 64, 8, 128, 6500, F16, E4M3, 64, "paged128"),
          (20, 24, 256, 64, 64, 2080, BF16, E4M3, 16, "paged64"), (5, 66, 32, 16, 128, 2100, F16, I8, 16, "shd")]


@pytest.mark.parametrize("B,T,hq,H,D,S,qt,cache,block,layout", SHARED)
@pytest.mark.parametrize("with_tree", [False, True])
def test_work_enough_for_shared_keys(B, T, hq, H, D, S, qt, cache, block, layout, with_tree):
    """Rows enough for a workgroup's waves to share keys, over ragged lengths, NaN
    behind them, absent pages, NaN that some queries see; some key/value heads
    compared, all of them from call to call."""
    q, k, v, ks, vs, table = make(B, T, hq, H, D, S, qt, cache, block, layout, seed=B + T + with_tree, dev=DEV)
    g = torch.Generator().manual_seed(B)
    G = hq // H
    length = torch.randint(S // 2, S - T, (B,), generator=g).to(torch.int32)
    drafted = torch.full((B,), T, dtype=torch.int32)
    if B > 1:
        length[0], length[1], drafted[1], drafted[2] = S - T, 0, T - 1, 0
    tree = None
    if with_tree:
        tree = torch.rand(B, T, T, generator=g) < 0.4
        tree |= torch.eye(T, dtype=torch.bool)
    if cache == E4M3 and table is None:
        for b in range(B):
            bits(k)[b, int(length[b]) + T:] = 0x7f
            bits(v)[b, int(length[b]) + T:] = 0x7f
        bits(v)[0, int(length[0]) + T - 1, :, 3] = 0x7f
    if table is not None:
        table[0, 1] = -1
        table[-1, -1] = k.shape[0] + 5
    at = sorted({0, H // 2, H - 1})
    heads = [h * G + i for h in at for i in range(G)]
    some = sorted({0, 1 % B, 2 % B, B - 1})
    got = []
    for _ in range(2):
        lse, w = torch.empty(B, T, hq, device=DEV), torch.zeros(B, H, k.shape[1] if table is None else table.shape[1] * k.shape[1], device=DEV)
        out = kv.attend(q, put(k.cpu(), layout), put(v.cpu(), layout), length.to(DEV), table=table, tree=put(tree), drafted=drafted.to(DEV), lse=lse, score=w,
                        k_scale=put(ks.cpu(), layout), v_scale=put(vs.cpu(), layout))
        got.append((out, lse, w))
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(*got))
    for b in some:
        # a few rows of each: the 64-bit form takes a row at a time
        rows = sorted({0, 1 % T, T // 2, T - 1})
        for h in at:
            args = [t[:, :, h:h + 1] for t in (k, v, ks, vs)] if table is not None else [t[b:b + 1, :, h:h + 1] for t in (k, v, ks, vs)]
            want = step_rows(q[b:b + 1, :, h * G:h * G + G].cpu(), [t.cpu() for t in args], block, length[b:b + 1],
                             None if table is None else table[b:b + 1].cpu(), None if tree is None else tree[b:b + 1], drafted[b:b + 1], rows, qt == BF16)
            for i, (o, ob, l, lb) in want.items():
                ref.within(out[b, i, h * G:h * G + G], o, ob, f"out {b} {i} {h}")
                ref.within(lse[b, i, h * G:h * G + G], l, lb, f"lse {b} {i} {h}")
    assert heads
    total = (drafted * hq).double()
    fine = torch.isfinite(w).all(-1).all(-1).cpu()
    assert ((w.double().sum((1, 2)).cpu() - total).abs() <= total * 2.0 ** -10)[fine & (length > 0)].all()


@pytest.mark.parametrize("B,T,hq,H,D,S,cache,block,layout", [
    (70, 1, 16, 8, 128, 4000, E4M3, 16, "shd"), (35, 3, 8, 4, 120, 9000, I8, 32, "paged64"), (130, 2, 8, 2, 128, 500, I8, 16, "paged16"),
    (300, 1, 8, 8, 64, 100, E4M3, 64, "shd"), (9, 5, 16, 1, 64, 3000, I8, 16, "hsd"), (66, 1, 1, 1, 256, 2500, E4M3, 16, "shd"),
    (700, 1, 8, 8, 128, 40, I8, 16, "shd"), (5, 20, 16, 8, 128, 5000, I8, 128, "shd"), (80, 9, 8, 2, 192, 300, E4M3, 16, "shd")])
def test_many_sequences(B, T, hq, H, D, S, cache, block, layout):
    """Ragged ones, some of nothing: runs of their own, shares of all sequences, a workgroup a sequence."""
    q, k, v, ks, vs, table = make(B, T, hq, H, D, S, BF16, cache, block, layout, seed=B + S, dev=DEV)
    g = torch.Generator().manual_seed(B)
    G = hq // H
    length = torch.randint(0, S - T + 1, (B,), generator=g).to(torch.int32)
    length[::7], length[1::9] = 0, S - T
    drafted = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    drafted[B // 2], length[B // 2] = T, S - T
    lse, w = torch.empty(B, T, hq, device=DEV), torch.zeros(B, H, k.shape[1] if table is None else table.shape[1] * k.shape[1], device=DEV)
    out = kv.attend(q, put(k.cpu(), layout), put(v.cpu(), layout), length.to(DEV), table=table, drafted=drafted.to(DEV), lse=lse, score=w,
                    k_scale=put(ks.cpu(), layout), v_scale=put(vs.cpu(), layout))
    for b in sorted({0, 1, 2, 5 % B, B // 2, B - 1, 63 % B, 64 % B, 65 % B}):
        for h in {0, H - 1}:
            args = [t[:, :, h:h + 1] for t in (k, v, ks, vs)] if table is not None else [t[b:b + 1, :, h:h + 1] for t in (k, v, ks, vs)]
            want = step_rows(q[b:b + 1, :, h * G:h * G + G].cpu(), [t.cpu() for t in args], block, length[b:b + 1],
                             None if table is None else table[b:b + 1].cpu(), None, drafted[b:b + 1], range(T), False)
            for i, (o, ob, l, lb) in want.items():
                ref.within(out[b, i, h * G:h * G + G], o, ob, f"out {b} {i} {h}")
                ref.within(lse[b, i, h * G:h * G + G], l, lb, f"lse {b} {i} {h}")
    total = (drafted * hq).double()
    assert ((w.double().sum((1, 2)).cpu() - total).abs() <= total * 2.0 ** -10).all()


def step_rows(q, args, block, length, table, tree, drafted, rows, coarse):
    """Rows of one sequence and key/value head by the 64-bit form, with their bounds."""
    k, v, ks, vs = args
    kk, vv = step.whole(k, ks, block), step.whole(v, vs, block)
    n, T = int(length[0]), q.shape[1]
    nd = int(drafted[0])
    cap = k.shape[1] if table is None else table.shape[1] * k.shape[1]
    end = min(n + nd, cap) if nd else 0
    kr, there = ref.rows_of(kk, table, 0, end)
    vr, _ = ref.rows_of(vv, table, 0, end)
    kr, vr = kr[:, 0], vr[:, 0]
    got = {}
    for i in rows:
        o, ob = torch.zeros(q.shape[2], q.shape[3], dtype=F64), torch.zeros(q.shape[2], q.shape[3], dtype=F64)
        l, lb = torch.full((q.shape[2],), -math.inf, dtype=F64), torch.zeros(q.shape[2], dtype=F64)
        see = there.clone()
        j = torch.arange(end) - n
        see &= (j < 0) | ((tree[0, i][j.clamp(0, T - 1)] if tree is not None else j <= i))
        if i < nd and bool(see.any()):
            for a in range(q.shape[2]):
                x = q[0, i, a].to(F64)
                s = kr[see] @ x / math.sqrt(q.shape[3])
                l[a] = torch.logsumexp(s, 0)
                p = torch.exp(s - l[a])
                o[a] = p @ vr[see]
                spread = p @ vr[see].abs()
                size = float((kr[see].abs() @ x.abs()).max()) / math.sqrt(q.shape[3])
                ds = (q.shape[3] + 16) * 2.0 ** -23 * size + 2.0 ** -21 * (1 + size)
                sums = int(see.sum()) * 2.0 ** -24
                ob[a] = ((2.0 ** -8 * (1 + 2.0 ** -7) if coarse else 2.0 ** -11) + 2 * ds + sums) * spread + ref.HALF[q.dtype] * (1 + 2.0 ** -7) * o[a].abs() + ref.TINY[q.dtype]
                lb[a] = 2 * ds + sums + 2.0 ** -22 * float(l[a].abs())
        got[i] = (o, ob, l, lb)
    return got


def test_attend_in_a_graph_on_another_stream():
    q, k, v, ks, vs, table = make(3, 4, 16, 2, 128, 900, cache=E4M3, layout="paged64", seed=5)
    n = torch.tensor([896, 30, 500], dtype=torch.int32, device=DEV)
    dq, dk, dv, dks, dvs, dt = (put(t) for t in (q, k, v, ks, vs, table))
    want = kv.attend(dq, dk, dv, n, table=dt, k_scale=dks, v_scale=dvs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kv.attend(dq, dk, dv, n, table=dt, k_scale=dks, v_scale=dvs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(dq)
    ws = torch.empty(kv.attend_workspace_bytes(3, 2, 128, 15 * 64, 4, 16, True), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend(dq, dk, dv, n, table=dt, k_scale=dks, v_scale=dvs, out=out, ws=ws)
    for _ in range(4):
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ----------------------------------------------------------------- append --
def new_tokens(B, T, H, D, dtype, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    mk = lambda: (torch.randn(B, T, H, D, generator=g) * torch.exp(spread * torch.randn(B, T, H, 1, generator=g))).to(dtype)  # noqa: E731
    return mk(), mk()


def powers(s):
    return torch.exp2(torch.floor(torch.log2(s)))


def check_append(B, T, H, D, S, dtype, cache, block, layout, length, drafted=None, seed=0, pow2=True, table_change=None, new=None, scale=1.0):
    """Without rotation everything is exact: elements and scales are equal, and nothing else is written."""
    _, k, v, ks, vs, table = make(B, 1, H, H, D, S, dtype, cache, block, layout, seed=seed)
    ks, vs = ks * scale, vs * scale
    if pow2:
        ks, vs = powers(ks), powers(vs)
    if table_change is not None:
        table_change(table)
    nk, nv = new or new_tokens(B, T, H, D, dtype, seed + 1)
    n = torch.tensor(length, dtype=torch.int32)
    d = None if drafted is None else torch.tensor(drafted, dtype=torch.int32)
    dk, dv, dks, dvs = put(k, layout), put(v, layout), put(ks, layout), put(vs, layout)
    assert kv.append(None, put(nk), put(nv), dk, dv, n.to(DEV), table=put(table), drafted=put(d), k_scale=dks, v_scale=dvs) is None
    for what, got, s, before, sb, x in (("k", dk, dks, k, ks, nk), ("v", dv, dvs, v, vs, nv)):
        want, ws, written = step.append8(before, sb, x.to(F64), n, d, table, block)
        assert torch.equal(s.cpu().to(F64), ws), what
        g = got.cpu()
        assert torch.equal(bits(g.contiguous())[~written], bits(before)[~written]), what
        a, b = g.to(F64)[written], want[written]
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)), what


@pytest.mark.parametrize("cache", [I8, E4M3])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,D,block", [(1, 128, 16), (1, 8, 32), (5, 64, 16), (33, 72, 16), (40, 128, 64), (100, 256, 32), (130, 200, 128), (17, 16, 16)])
def test_append_is_exact(cache, dtype, T, D, block):
    check_append(3, T, 2, D, T + 60, dtype, cache, block, "shd", [0, 27, 60], seed=T)


@pytest.mark.parametrize("layout,block", [("hsd", 16), ("paged16", 16), ("paged64", 16), ("paged64", 64), ("paged128", 32)])
@pytest.mark.parametrize("cache", [I8, E4M3])
def test_append_layouts_and_ends(layout, block, cache):
    """Past the capacity, before the first token, fewer than given, none, absent pages."""
    def holes(table):
        if table is not None:
            table[1, 0] = -1
            table[4, -1] = 10 ** 6
    check_append(6, 21, 3, 64, 256, BF16, cache, block, layout, [0, 5, 250, -7, 240, 300], [21, 21, 30, 21, 9, 21], seed=6, table_change=holes)
    check_append(6, 21, 3, 64, 256, BF16, cache, block, layout, [16, 31, 33, 100, 127, 128], [0, 1, -3, 16, 17, 21], seed=7)


@pytest.mark.parametrize("cache", [I8, E4M3])
def test_scales_that_are_no_powers_of_two(cache):
    """Kept where they hold the new tokens; else earlier tokens are rounded anew, by a ratio in binary32."""
    kept = grown = 0
    for times in (1.0, 8.0):
        _, k, v, ks, vs, _ = make(2, 1, 4, 4, 64, 64, BF16, cache, 16, seed=3)
        ks, vs = ks * times, vs * times
        nk, nv = new_tokens(2, 6, 4, 64, BF16, 5)
        n = torch.tensor([20, 40], dtype=torch.int32)
        dk, dv, dks, dvs = (put(t) for t in (k, v, ks, vs))
        kv.append(None, put(nk), put(nv), dk, dv, n.to(DEV), k_scale=dks, v_scale=dvs)
        for got, s, before, sb, x in ((dk, dks, k, ks, nk), (dv, dvs, v, vs, nv)):
            want, ws, written = step.append8(before, sb, x.to(F64), n, None, None, 16)
            assert torch.equal(s.cpu().to(F64), ws)
            kept += int((ws == sb.to(F64))[0, 1].sum())
            grown += int((ws != sb.to(F64))[0, 1].sum())
            # a product of 24 bits before the rounding: at a border the other neighbour, a step away
            a, b = got.cpu().to(F64)[written], want[written]
            one = torch.ones_like(b) if cache == I8 else b.abs().clamp(min=2.0 ** -6) * 2.0 ** -3
            assert ((a - b).abs() <= one).all() and ((a != b).double().mean() < 1e-3)
    assert kept and grown


@pytest.mark.parametrize("cache", [I8, E4M3])
def test_values_that_are_not_finite_and_zeros(cache):
    nk, nv = new_tokens(2, 20, 2, 64, BF16, 9)
    nk[0, 3, 0, 5], nk[0, 4, 0, 6], nk[0, 5, 1, 7], nv[1, 2, 1] = math.inf, -math.inf, math.nan, math.nan
    nk[1, :, 0], nv[0, 16:] = 0.0, 0.0
    nk[1, 17, 1], nv[1, 3, 0, 0] = 2.0 ** -90, 3e38
    check_append(2, 20, 2, 64, 40, BF16, cache, 16, "shd", [0, 16], new=(nk, nv))


def test_a_scale_grows_once():
    """One token at a time, ever larger: earlier ones stay within half a step of the largest scale and one rounding each growth."""
    H, D = 2, 64
    k, v = (torch.zeros(1, 16, H, D, dtype=I8, device=DEV) for _ in "kv")
    ks, vs = (torch.full((1, 1, H), math.nan, device=DEV) for _ in "kv")
    x = torch.randn(1, 16, H, D, generator=torch.Generator().manual_seed(1)).to(BF16) * torch.exp2(torch.arange(16) // 3)[None, :, None, None]
    x = x.to(BF16)
    for t in range(16):
        kv.append(None, x[:, t:t + 1].to(DEV), -x[:, t:t + 1].to(DEV), k, v, torch.tensor([t], dtype=torch.int32, device=DEV), k_scale=ks, v_scale=vs)
    assert torch.equal(k, -v) and torch.equal(ks, vs) and torch.equal(powers(ks), ks)
    s = ks.cpu().to(F64)[0, 0]
    off = (k.cpu().to(F64) * s[None, None, :, None] - x.to(F64)).abs()
    # halves of s, s / 2, s / 4, ...: together below s
    assert (off <= s[None, None, :, None]).all()
    assert (x.abs().amax((1, 3))[0].to(F64) <= s * 127).all() and (x.abs().amax((1, 3))[0].to(F64) > s * 127 / 2).all()


@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (F16, I8), (BF16, I8)])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 20, False), (72, 20, True), (256, 256, False), (64, 0, False), (80, 16, False)])
@pytest.mark.parametrize("T", [1, 37])
def test_append_turns(dtype, cache, D, rot, interleaved, T):
    """Queries as kv.rope's; keys within half a step of the 64-bit form and what binary32 loses on the way."""
    B, H, hq, block = 2, 2, 6, 32
    _, k, v, ks, vs, _ = make(B, 1, H, H, D, 100, dtype, cache, block, seed=D)
    k, v = torch.zeros_like(bits(k)).view(cache), torch.zeros_like(bits(v)).view(cache)
    nk, nv = new_tokens(B, T, H, D, dtype, D + T)
    q = torch.randn(B, T, hq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    n = torch.tensor([0, 64], dtype=torch.int32)
    pos = torch.tensor([[5], [10 ** 6]], dtype=torch.int32) + torch.arange(T, dtype=torch.int32)
    freq = kv.rope_freq(rot, 1000.0) if rot else None
    for at in (None, pos):
        where = n[:, None] + torch.arange(T) if at is None else at
        dk, dv, dks, dvs = (put(t) for t in (k, v, ks, vs))
        kw = dict(amplitude=1.25, interleaved=interleaved, pos=put(at)) if rot else {}
        got = kv.append(put(q), put(nk), put(nv), dk, dv, n.to(DEV), put(freq), k_scale=dks, v_scale=dvs, **kw)
        if rot:
            want = ref.turned(q, where, freq, 1.25, interleaved)
            ref.within(got, want, ref.rope_bound(q, want, freq, 1.25, dtype), "q")
            xk = ref.turned(nk, where, freq, 1.25, interleaved)
        else:
            assert torch.equal(got.cpu(), q)
            xk = nk.to(F64)
        inplace = put(q)
        dk2, dv2, dks2, dvs2 = (put(t) for t in (k, v, ks, vs))
        kv.append(inplace, put(nk), put(nv), dk2, dv2, n.to(DEV), put(freq), k_scale=dks2, v_scale=dvs2, out=inplace, **kw)
        assert torch.equal(dk, dk2) and torch.equal(dv, dv2) and torch.equal(dks, dks2)
        if rot:
            ref.within(inplace, want, ref.rope_bound(q, want, freq, 1.25, dtype), "q in place")
        for x, c, s in ((xk, dk, dks), (nv.to(F64), dv, dvs)):
            for b in range(B):
                lo, m = int(n[b]), min(T, 100 - int(n[b]))     # the last of 37 tokens is behind the end
                rows, xb = c[b, lo:lo + m].cpu().to(F64), x[b, :m]
                sc = s[b].cpu().to(F64).repeat_interleave(block, 0)[lo:lo + m, :, None]
                y = xb / sc
                slip = xb.abs().amax(-1, keepdim=True) * 2.0 ** -20 / sc
                half = torch.full_like(y, 0.5) if cache == I8 else torch.maximum(y.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=F64))
                assert ((rows - y).abs() <= half * (1 + 2.0 ** -10) + slip).all()
                for first in range(lo // block * block, lo + m, block):
                    part = xb[max(first - lo, 0):first + block - lo].abs().amax((0, 2))
                    sb = s[b, first // block].cpu().to(F64)
                    assert torch.equal(powers(sb), sb)
                    assert (part <= sb * MOST[cache] * (1 + 2.0 ** -20)).all() and (part > sb / 2 * MOST[cache] * (1 - 2.0 ** -20)).all()


@pytest.mark.parametrize("D", [256, 128, 120])
def test_many_angles_in_a_block(D):
    """More than a workgroup holds, worked out where they are used, and as many as it holds."""
    block, T = 128, 128
    nk, nv = new_tokens(1, T, 1, D, BF16, 3)
    freq = kv.rope_freq(D, device=DEV)
    got = []
    for b in (block, 16):
        k, v = (torch.zeros(1, T, 1, D, dtype=E4M3, device=DEV) for _ in "kv")
        ks, vs = (torch.zeros(1, T // b, 1, device=DEV) for _ in "kv")
        kv.append(None, put(nk), put(nv), k, v, torch.zeros(1, dtype=torch.int32, device=DEV), freq, k_scale=ks, v_scale=vs)
        got.append(step.whole(k.cpu(), ks.cpu(), b))
    want = ref.turned(nk, torch.arange(T)[None], freq.cpu())
    for g in got:
        assert ((g - want).abs() <= want.abs() * 2.0 ** -4 * (1 + 2.0 ** -9) + want.abs().max() * 2.0 ** -18).all()


def test_append_then_attend_in_a_graph():
    """A step as a server captures it, replayed: the same cache and output each time."""
    B, T, hq, H, D = 3, 4, 16, 2, 128
    _, k, v, ks, vs, table = make(B, 1, H, H, D, 200, BF16, I8, 16, "paged32", seed=2)
    ks, vs = powers(ks), powers(vs)
    nk, nv = (put(t) for t in new_tokens(B, T, H, D, BF16, 1))
    q = torch.randn(B, T, hq, D, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    freq = kv.rope_freq(D, device=DEV)
    n = torch.tensor([190, 0, 77], dtype=torch.int32, device=DEV)
    dk, dv, dks, dvs, dt = (put(t) for t in (k, v, ks, vs, table))
    turned, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(kv.attend_workspace_bytes(B, H, D, 7 * 32, T, hq, True), dtype=torch.uint8, device=DEV)

    def run():
        kv.append(q, nk, nv, dk, dv, n, freq, table=dt, k_scale=dks, v_scale=dvs, out=turned)
        kv.attend(turned, dk, dv, n, table=dt, k_scale=dks, v_scale=dvs, out=out, ws=ws)
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dk, dv, dks, dvs, turned, out)]
    full = step.attend8(turned.cpu(), dk.cpu(), dv.cpu(), dks.cpu(), dvs.cpu(), 16, n.cpu(), table=table)
    ref.within(out, full["out"], full["out_bound"], "out")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t, w in ((dk, put(k)), (dv, put(v)), (dks, put(ks)), (dvs, put(vs))):
            t.copy_(w)
        out.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dk, dv, dks, dvs, turned, out), want))
