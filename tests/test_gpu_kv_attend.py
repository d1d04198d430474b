"""kv.attend against its 64-bit form: types, head layouts, lengths, trees,
pages, masked values that are not finite, and the ways it is called."""
import math

import pytest
import torch

import kv_reference as ref
from lossless_bf16_tensor_amd import kv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, E5M2 = torch.bfloat16, torch.float16, torch.float8_e5m2


def bits(t):
    return t.view(torch.uint8) if t.dtype == E5M2 else t


def make(B, T, hq, H, D, S, q=BF16, cache=None, layout="shd", seed=0, kscale=1.0):
    """q, k, v, table on the CPU; caches with noise everywhere."""
    g = torch.Generator().manual_seed(seed)
    cache = cache or q
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    qq = mk(B, T, hq, D).to(q)
    if layout.startswith("paged"):
        page = int(layout[5:])
        per = -(-S // page)
        pool = B * per + 2
        k, v = (mk(pool, page, H, D) * kscale).to(cache), mk(pool, page, H, D).to(cache)
        table = torch.randperm(pool, generator=g)[:B * per].view(B, per).to(torch.int32)
        return qq, k, v, table
    k, v = (mk(B, S, H, D) * kscale).to(cache), mk(B, S, H, D).to(cache)
    return qq, k, v, None


def put(t, layout="shd"):
    if t is None:
        return None
    if layout == "hsd":
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    return t.to(DEV)


def check(q, k, v, length, table=None, tree=None, drafted=None, layout="shd", scale=None, score=True, **kw):
    B, T, hq, D = q.shape
    cap = k.shape[1] if table is None else table.shape[1] * k.shape[1]
    length = torch.tensor(length, dtype=torch.int32)
    drafted = None if drafted is None else torch.tensor(drafted, dtype=torch.int32)
    want = ref.attend(q, k, v, length, table=table, tree=tree, drafted=drafted, scale=scale)
    lse = torch.full((B, T, hq), 7.0, device=DEV)
    w = torch.full((B, k.shape[2], cap), 0.25, device=DEV) if score else None
    out = kv.attend(put(q), put(k, layout), put(v, layout), length.to(DEV), table=put(table),
                    tree=put(tree), drafted=put(drafted), scale=scale, score=w, lse=lse, **kw)
    ref.within(out, want["out"], want["out_bound"], "out")
    ref.within(lse, want["lse"], want["lse_bound"], "lse")
    if score:
        ref.within(w, want["weight"] + 0.25, want["weight_bound"] + 2.0 ** -24 * (want["weight"] + 0.25), "score")
    return out, lse, w


@pytest.mark.parametrize("n", [0, 1, 14, 15, 16, 30, 31, 32, 33, 63, 64, 100, 257, 1000, 2500])
def test_one_token(n):
    q, k, v, _ = make(1, 1, 8, 2, 128, n + 1, seed=n)
    check(q, k, v, [n])


@pytest.mark.parametrize("q,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2), (F16, E5M2)])
@pytest.mark.parametrize("D", [8, 16, 64, 72, 128, 200, 256])
def test_types_and_head_dims(q, cache, D):
    for T, hq, H in ((1, 6, 2), (7, 8, 2), (21, 10, 5)):
        a, k, v, _ = make(2, T, hq, H, D, 150 + T, q, cache, seed=D + T)
        check(a, k, v, [150, 61], drafted=[T, T])


@pytest.mark.parametrize("T,hq,H", [(1, 1, 1), (2, 7, 1), (17, 1, 1), (5, 16, 2), (9, 14, 2), (16, 8, 2), (33, 8, 2),
                                    (65, 4, 1), (40, 32, 4), (130, 3, 1)])
def test_row_counts(T, hq, H):
    """From one row a key/value head to several workgroups of rows."""
    q, k, v, _ = make(1, T, hq, H, 64, 200 + T, seed=T)
    check(q, k, v, [200])
    q, k, v, _ = make(1, T, hq, H, 256, 40 + T, seed=T + 1)
    check(q, k, v, [37])


@pytest.mark.parametrize("layout", ["shd", "hsd", "paged16", "paged32", "paged128"])
@pytest.mark.parametrize("cache", [BF16, E5M2])
def test_layouts_and_ragged_lengths(layout, cache):
    B, T, S = 5, 4, 300
    q, k, v, table = make(B, T, 8, 4, 128, S, BF16, cache, layout, seed=3)
    check(q, k, v, [296, 0, 1, 100, 250], table=table, drafted=[4, 4, 0, 3, 1], layout=layout)


def tree_of(T, seed, B=None):
    g = torch.Generator().manual_seed(seed)
    shape = (T, T) if B is None else (B, T, T)
    return torch.rand(*shape, generator=g) < 0.3


@pytest.mark.parametrize("T", [1, 2, 13, 32, 33, 70])
@pytest.mark.parametrize("n", [0, 5, 64, 90])
def test_trees(T, n):
    """Any mask, rows that see no drafted token and (n = 0) nothing at all among them."""
    q, k, v, _ = make(2, T, 4, 2, 128, n + T, seed=T + n)
    tree = tree_of(T, T, 2)
    tree[:, T // 2] = False
    out, lse, _ = check(q, k, v, [n, n], tree=tree, drafted=[T, max(0, T - 2)])
    if n == 0:
        assert not out[:, T // 2].any() and torch.isinf(lse[:, T // 2]).all()


def test_one_tree_for_all_and_bytes():
    q, k, v, table = make(3, 9, 6, 3, 80, 120, layout="paged16", seed=5)
    tree = tree_of(9, 1)
    a = check(q, k, v, [100, 3, 0], table=table, tree=tree)
    b = check(q, k, v, [100, 3, 0], table=table, tree=tree.to(torch.uint8) * 255)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2)])
@pytest.mark.parametrize("T,hq", [(6, 4), (20, 8), (40, 8)])
def test_masked_values_have_no_effect(dtype, cache, T, hq):
    """Infinities and NaN in keys and values that some queries do not see, and in memory behind the last token."""
    n = 45
    q, k, v, _ = make(1, T, hq, 2, 64, n + T + 40, dtype, cache, seed=T)
    tree = torch.eye(T, dtype=torch.bool)
    tree[:, 0] = True
    for t, bad in ((k, math.nan), (v, math.inf)):
        bits(t)[:, n + 2] = bits(torch.full((1,), bad).to(cache))
    bits(v)[:, n + 4, :, 5] = bits(torch.full((1,), math.nan).to(cache))
    for t in (k, v):
        bits(t)[:, n + T:] = bits(torch.full((1,), math.nan).to(cache))
    out, lse, _ = check(q, k, v, [n], tree=tree)
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2]).all()
    assert torch.isnan(out[0, 4, :, 5]).all() and not torch.isnan(out[0, 4, :, 6]).any()
    assert not torch.isnan(out[0, 5]).any()


def test_scores_at_the_ends():
    """A seen key of -inf everywhere gives zeros; one of +inf or NaN gives NaN; large scores do not overflow."""
    q, k, v, _ = make(4, 1, 2, 1, 64, 40, seed=9)
    q[:, :, :, 0] = 1.0
    k[0, :, :, 0] = -math.inf
    k[1, 7, :, 0] = math.inf
    k[2, 9, :, 3] = math.nan
    k[3] *= 1e4
    out, lse, _ = check(q, k, v, [39, 39, 39, 39])
    assert not out[0].any() and torch.isnan(out[1]).all() and torch.isnan(out[2]).all() and torch.isfinite(out[3]).all()


def test_fp8_cache_with_large_and_small_queries():
    """Queries far outside FP16's range: their rows are scaled by a power of two."""
    q, k, v, _ = make(1, 4, 4, 2, 128, 100, BF16, E5M2, seed=4)
    q[:, 0] *= 2.0 ** 90
    q[:, 1] *= 2.0 ** -100
    q[:, 2, :, 5] *= 2.0 ** 20
    k = (k.float() * 2.0 ** -14).to(E5M2)         # subnormal keys among them
    check(q[:, 1:], k, v, [96])
    check(q[:, :1], k, v, [96], scale=2.0 ** -60)


def test_absent_pages():
    """Table entries outside the pool: their tokens are not there."""
    q, k, v, table = make(2, 3, 4, 2, 128, 200, layout="paged16", seed=8)
    table[0, 3] = -1
    table[0, 12] = 1 << 30
    table[1, :] = -7
    check(q, k, v, [190, 190], table=table)


def test_score_shorter_than_the_pages():
    q, k, v, table = make(2, 5, 4, 2, 64, 75, layout="paged32", seed=8)
    n = torch.tensor([70, 20], dtype=torch.int32)
    want = ref.attend(q, k, v, n, table=table)
    whole = torch.zeros(2, 2, 80, device=DEV)
    out = kv.attend(put(q), put(k), put(v), n.to(DEV), table=put(table), score=whole[..., :73])
    ref.within(out, want["out"], want["out_bound"])
    ref.within(whole[..., :73], want["weight"][..., :73], want["weight_bound"][..., :73])
    assert not whole[..., 73:].any()


def test_lengths_outside_the_cache_are_clamped():
    q, k, v, _ = make(4, 3, 4, 2, 64, 50, seed=2)
    check(q, k, v, [-5, 49, 50, 2 ** 31 - 1], drafted=[3, 3, 2, 9])


def test_strided_views():
    """Queries and caches inside larger tensors, a head dim that is a slice, outputs given."""
    g = torch.Generator().manual_seed(1)
    big = torch.randn(2, 70, 3, 2, 160, generator=g).to(BF16)          # tokens, (k, v, -), heads, dim
    k, v = big[:, :, 0, :, 16:144], big[:, :, 1, :, 16:144]
    q = torch.randn(2, 8, 5, 144, generator=g).to(BF16).transpose(1, 2)[..., :128]
    length = torch.tensor([60, 33], dtype=torch.int32)
    want = ref.attend(q, k, v, length)
    dbig = big.to(DEV)
    dq = torch.empty(2, 8, 5, 144, dtype=BF16, device=DEV)[..., :128].transpose(1, 2)
    dq.copy_(q)
    whole = torch.full((2, 5, 8, 136), 3.0, dtype=BF16, device=DEV)
    got = kv.attend(dq, dbig[:, :, 0, :, 16:144], dbig[:, :, 1, :, 16:144], length.to(DEV), out=whole[..., :128])
    ref.within(got, want["out"], want["out_bound"])
    assert (whole[..., 128:] == 3.0).all()


def test_long_rows_are_split_and_joined():
    q, k, v, table = make(1, 2, 4, 1, 128, 40000, BF16, E5M2, "paged64", seed=6)
    check(q, k, v, [39990], table=table, drafted=[2])


def test_far_rows_of_a_large_cache():
    """Offsets past 32 bits: the last page of a pool of 4.8 GB."""
    page, H, D, n = 1 << 10, 3, 128, 70
    g = torch.Generator().manual_seed(0)
    k, v = (torch.empty(6 << 10, page, H, D, dtype=BF16, device=DEV) for _ in range(2))
    rows = torch.randn(2, 1, n + 1, H, D, generator=g).to(BF16)
    k[-1, :n + 1], v[-1, :n + 1] = rows[0, 0].to(DEV), rows[1, 0].to(DEV)
    q = torch.randn(1, 1, H, D, generator=g).to(BF16)
    length = torch.tensor([n], dtype=torch.int32)
    want = ref.attend(q, rows[0], rows[1], length)
    table = torch.full((1, 1), k.shape[0] - 1, dtype=torch.int32, device=DEV)
    got = kv.attend(q.to(DEV), k, v, length.to(DEV), table=table)
    ref.within(got, want["out"], want["out_bound"])


def test_same_result_every_time_and_in_any_workspace():
    q, k, v, _ = make(2, 12, 8, 2, 128, 3000, seed=7)
    dq, dk, dv, n = put(q), put(k), put(v), torch.tensor([2900, 1234], dtype=torch.int32, device=DEV)
    ws = torch.empty(kv.attend_workspace_bytes(2, 2, 128, 3000, 12, 8), dtype=torch.uint8, device=DEV)
    first = None
    for fill in (0, 255, 127, 0):
        ws.fill_(fill)
        w, lse = torch.zeros(2, 2, 3000, device=DEV), torch.zeros(2, 12, 8, device=DEV)
        got = (kv.attend(dq, dk, dv, n, score=w, lse=lse, ws=ws), lse, w)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    # the weights of a query add up to one
    assert torch.allclose(first[2].sum(-1), torch.full((2, 2), 12.0 * 4, device=DEV), rtol=1e-4)


def test_on_streams_and_in_a_graph():
    q, k, v, _ = make(2, 3, 8, 2, 128, 1500, seed=11)
    dq, dk, dv, n = put(q), put(k), put(v), torch.tensor([1400, 700], dtype=torch.int32, device=DEV)
    want = ref.attend(q, k, v, n.cpu())
    eager = kv.attend(dq, dk, dv, n)
    ref.within(eager, want["out"], want["out_bound"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [kv.attend(dq, dk, dv, n, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, eager) for g in got)

    score = torch.zeros(2, 2, 1500, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.attend(dq, dk, dv, n, score=score)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kv.attend(dq, dk, dv, n, score=score)
    for lens in ([1400, 700], [1, 1499], [0, 64], [1400, 700]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9.0)
        score.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        w = torch.zeros_like(score)
        assert torch.equal(out, kv.attend(dq, dk, dv, n, score=w)) and torch.equal(score, w)


@pytest.mark.parametrize("layout,D,cache", [("paged16", 128, BF16), ("paged32", 64, E5M2), ("paged128", 72, F16), ("paged16", 72, E5M2),
                                            ("hsd", 128, E5M2), ("hsd", 40, E5M2), ("shd", 96, BF16)])
@pytest.mark.parametrize("T,hq,H", [(9, 8, 2), (20, 8, 2), (37, 4, 1), (70, 4, 1)])
def test_many_rows_over_ragged_caches(layout, D, cache, T, hq, H):
    """Rows that share keys: ends inside tiles and pages, absent pages, sequences of nothing between others."""
    S = 900
    q, k, v, table = make(5, T, hq, H, D, S, F16 if cache == F16 else BF16, cache, layout, seed=T + D)
    if table is not None:
        page = k.shape[1]
        table[0, 160 // page] = -1
        table[0, 700 // page] = 1 << 28
        table[4, :3] = k.shape[0]
    tree = tree_of(T, 4, 5)
    tree[:, 3] = False
    lens = dict(length=[S - T, 0, 33, 511, 640], drafted=[T, 0, T, T - 1, 1], table=table, layout=layout)
    check(q, k, v, **lens)
    check(q, k, v, tree=tree, **lens)


@pytest.mark.parametrize("B,layout", [(3, "shd"), (64, "shd"), (65, "paged16"), (200, "shd"), (1100, "paged32")])
def test_many_sequences_of_many_rows(B, layout):
    """Lengths of every size side by side, those of nothing too; some of the sequences compared."""
    T, hq, H, D, S = 5, 8, 1, 64, 400
    q, k, v, table = make(B, T, hq, H, D, S, layout=layout, seed=B)
    g = torch.Generator().manual_seed(B)
    length = torch.randint(0, S - T, (B,), generator=g).to(torch.int32)
    length[::7] = 0
    length[1::9] = 3
    drafted = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    drafted[B // 2] = T
    w, lse = torch.zeros(B, H, k.shape[1] if table is None else table.shape[1] * k.shape[1], device=DEV), torch.empty(B, T, hq, device=DEV)
    out = kv.attend(put(q), put(k), put(v), length.to(DEV), table=put(table), drafted=drafted.to(DEV), score=w, lse=lse)
    at = sorted({0, 1, 2, B // 2, B - 1, 63 % B, 64 % B})
    want = ref.attend(q[at], *((k[at], v[at]) if table is None else (k, v)), length[at], table=None if table is None else table[at], drafted=drafted[at])
    for name, got in (("out", out), ("lse", lse), ("weight", w)):
        ref.within(got[at], want[name], want[name + "_bound"], name)
    # the others: each alone, whose splits differ; and the weights' sum
    total = (drafted * hq).double()
    assert ((w.double().sum((1, 2)).cpu() - total).abs() <= total * 2.0 ** -10).all()
    for b in range(0, B, max(1, B // 8)):
        alone = kv.attend(put(q[b:b + 1]), *((put(k[b:b + 1]), put(v[b:b + 1])) if table is None else (put(k), put(v))), length[b:b + 1].to(DEV),
                          table=None if table is None else put(table[b:b + 1]), drafted=drafted[b:b + 1].to(DEV))
        one = ref.attend(q[b:b + 1], *((k[b:b + 1], v[b:b + 1]) if table is None else (k, v)), length[b:b + 1],
                         table=None if table is None else table[b:b + 1], drafted=drafted[b:b + 1])
        ref.within(alone, one["out"], one["out_bound"], "alone")
        ref.within(out[b:b + 1], one["out"], one["out_bound"], "out")


@pytest.mark.parametrize("T,hq,H,D,n", [(6, 4, 2, 128, 3001), (40, 4, 1, 64, 3001), (40, 4, 1, 128, 2990), (24, 8, 1, 256, 1001)])
@pytest.mark.parametrize("cache", [BF16, E5M2])
def test_masked_values_in_split_rows(T, hq, H, D, n, cache):
    """Infinities that some queries see, in both signs, where the key axis is cut."""
    q, k, v, _ = make(1, T, hq, H, D, n + T, BF16, cache, seed=T + D)
    tree = torch.eye(T, dtype=torch.bool)
    tree[2, 3] = True
    for j, d, value in ((2, 0, math.inf), (3, 0, -math.inf), (3, 7, -math.inf), (4, 9, math.nan), (T - 1, 11, math.inf)):
        bits(v)[:, n + j, :, d] = bits(torch.full((1,), value).to(cache))
    out, _, _ = check(q, k, v, [n], tree=tree)
    assert torch.isnan(out[0, 2, :, 0]).all() and (out[0, 2, :, 7] == -math.inf).all() and (out[0, 3, :, 0] == -math.inf).all()
    assert torch.isnan(out[0, 4, :, 9]).all() and torch.isfinite(out[0, 5:T - 1]).all()


@pytest.mark.parametrize("D,cache", [(64, F16), (256, BF16), (200, E5M2)])
def test_weights_of_many_rows(D, cache):
    """More rows than the weights' kernel holds at once."""
    q, k, v, _ = make(2, 75, 8, 2, D, 330, F16 if cache == F16 else BF16, cache, seed=D)
    check(q, k, v, [255, 0], drafted=[75, 70])


def test_a_long_chain():
    q, k, v, _ = make(1, 300, 2, 1, 128, 520, seed=1)
    check(q, k, v, [211])


def test_many_rows_over_a_long_cache():
    """One sequence on every workgroup: more parts than a few lanes join."""
    q, k, v, _ = make(1, 10, 4, 1, 64, 33000, seed=2)
    check(q, k, v, [32985])


def test_two_graphs_at_once():
    """Each with a workspace and outputs of its own, replayed side by side."""
    T, S = 24, 2500
    q, k, v, _ = make(2, T, 8, 2, 128, S, seed=12)
    dq, dk, dv = put(q), put(k), put(v)
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([2400, 100], [64, 2300])]
    tree = put(tree_of(T, 3))
    want = []
    for n in lens:
        w = torch.zeros(2, 2, S, device=DEV)
        want.append((kv.attend(dq, dk, dv, n, tree=tree, score=w), w))
    graphs, got = [], []
    for n in lens:
        w = torch.zeros(2, 2, S, device=DEV)
        ws = torch.empty(kv.attend_workspace_bytes(2, 2, 128, S, T, 8), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(dq)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.attend(dq, dk, dv, n, tree=tree, score=w, out=out, ws=ws)
        graphs.append(g)
        got.append((out, w))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for out, w in got:
            out.fill_(5.0)
            w.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def large(B, T, hq, H, D, S, cache, layout, seed):
    """q, k, v, table on the device, as make() has them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q = mk(B, T, hq, D).to(F16 if cache == F16 else BF16)
    if layout.startswith("paged"):
        page = int(layout[5:])
        per = -(-S // page)
        k, v = (mk(B * per + 2, page, H, D).to(cache) for _ in range(2))
        return q, k, v, torch.randperm(B * per + 2, generator=g, device=DEV)[:B * per].view(B, per).to(torch.int32)
    shape = (B, H, S, D) if layout == "hsd" else (B, S, H, D)
    k, v = (mk(*shape).to(cache) for _ in range(2))
    return (q, k.transpose(1, 2), v.transpose(1, 2), None) if layout == "hsd" else (q, k, v, None)


SHARED = [(5, 24, 96, 32, 128, 1760, BF16, "shd"), (5, 70, 32, 8, 128, 2400, BF16, "paged16"), (5, 70, 32, 8, 64, 2400, E5M2, "paged32"),
          (5, 24, 96, 32, 72, 1760, F16, "hsd"), (5, 33, 64, 32, 48, 1800, E5M2, "hsd"), (1, 64, 64, 8, 128, 6500, BF16, "paged128"),
          (100, 24, 32, 8, 64, 2080, BF16, "shd"), (20, 24, 256, 64, 64, 2080, F16, "paged64"), (5, 66, 32, 16, 128, 2100, E5M2, "shd")]


@pytest.mark.parametrize("B,T,hq,H,D,S,cache,layout", SHARED)
@pytest.mark.parametrize("with_tree", [False, True])
def test_work_enough_for_shared_keys(B, T, hq, H, D, S, cache, layout, with_tree):
    """Rows enough for a workgroup's waves to share keys, over lengths of every
    size, NaN behind them, absent pages, infinities that some queries see; some
    key/value heads compared, all of them from call to call."""
    q, k, v, table = large(B, T, hq, H, D, S, cache, layout, B + T + with_tree)
    g = torch.Generator().manual_seed(B)
    G = hq // H
    length = torch.randint(S // 2, S - T, (B,), generator=g).to(torch.int32)
    drafted = torch.full((B,), T, dtype=torch.int32)
    if B > 1:
        length[1], length[2], drafted[2], drafted[B - 1] = 0, 77, 0, 3
        length[3] = S - T
    if table is None:
        for t in (k, v):
            for b in range(B):
                bits(t)[b, int(length[b]) + int(drafted[b]):] = bits(torch.full((1,), math.nan).to(cache)).to(DEV)
        bits(v)[0, int(length[0]) + 1, :, 1] = bits(torch.full((1,), math.inf).to(cache)).to(DEV)
    else:
        table[0, 300 // k.shape[1]] = -1
        table[B - 1, :2] = k.shape[0]
    tree = None
    if with_tree:
        tree = torch.rand(B, T, T, generator=g) < 0.2
        tree[:, 4] = False
    kw = dict(table=table, tree=put(tree), drafted=drafted.to(DEV))
    ws = torch.empty(kv.attend_workspace_bytes(B, H, D, S if table is None else table.shape[1] * k.shape[1], T, hq), dtype=torch.uint8, device=DEV)
    first = None
    for fill in (0, 255):
        ws.fill_(fill)
        w, lse = torch.zeros(B, H, S, device=DEV), torch.full((B, T, hq), 3.0, device=DEV)
        got = (kv.attend(q, k, v, length.to(DEV), score=w, lse=lse, ws=ws, **kw), lse, w)
        first = first or got
        assert all(torch.equal(a.nan_to_num(nan=-9.0), b.nan_to_num(nan=-9.0)) for a, b in zip(first, got))
    out, lse, w = got
    for b, h in {(0, 0), (min(1, B - 1), H - 1), (min(2, B - 1), 1), (B - 1, H // 2)}:
        at, heads = slice(b, b + 1), slice(h * G, h * G + G)
        one = (k[at, :, h:h + 1], v[at, :, h:h + 1]) if table is None else (k[:, :, h:h + 1], v[:, :, h:h + 1])
        want = ref.attend(q[at, :, heads].cpu(), *(t.cpu() for t in one), length[at], table=None if table is None else table[at].cpu(),
                          tree=None if tree is None else tree[at], drafted=drafted[at])
        ref.within(out[at, :, heads], want["out"], want["out_bound"], f"out {b} {h}")
        ref.within(lse[at, :, heads], want["lse"], want["lse_bound"], f"lse {b} {h}")
        ref.within(w[at, h:h + 1], want["weight"][..., :S], want["weight_bound"][..., :S], f"score {b} {h}")


def test_shared_keys_in_a_graph():
    q, k, v, _ = large(16, 24, 32, 8, 64, 2200, BF16, "shd", 1)
    n = torch.full((16,), 2000, dtype=torch.int32, device=DEV)
    kv.attend(q, k, v, n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kv.attend(q, k, v, n)
    for i in range(4):
        n.copy_((torch.arange(16) * 137 * i).clamp(max=2176).to(torch.int32))
        out.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kv.attend(q, k, v, n))
