"""kv.verify, kv.accept, kv.fork, kv.compact and kv.copy_pages against their plain forms."""
import math
import random

import pytest
import torch

import kv_step_reference as step
from lossless_bf16_tensor_amd import kv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def put(t):
    return None if t is None else t.to(DEV)


# ----------------------------------------------------------------- verify --
def problem(B, T, V, dtype=F32, draft=True, tree=False, seed=0, near=0.6, wide=3):
    g = torch.Generator().manual_seed(seed)
    logits = 2.0 * torch.randn(B, T, V, generator=g)
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits + near * torch.randn(B, T, V, generator=g), -1).to(dtype)
    rng = random.Random(seed)
    parent = None
    if tree:
        parent = torch.tensor([[-1] + [rng.randint(max(0, i // wide - 1), min(i - 1, i // wide)) for i in range(1, T)] for _ in range(B)], dtype=I32)
    tokens = torch.zeros(B, T, dtype=I32)
    for b in range(B):
        for i in range(1, T):
            up = i - 1 if parent is None else int(parent[b, i])
            tokens[b, i] = int(torch.multinomial(q[b, up].float(), 1, generator=g))
    return dict(tokens=tokens, target=p, uniform=torch.rand(B, T, generator=g), draft=q if draft else None, parent=parent)


def check(s, drafted=None, **kw):
    d = None if drafted is None else torch.tensor(drafted, dtype=I32)
    path, count, token = kv.verify(put(s["tokens"]), put(s["target"]), put(s["uniform"]), draft=put(s["draft"]), parent=put(s["parent"]), drafted=put(d), **kw)
    want = step.verify(s["tokens"], s["target"], s["uniform"], s["draft"], s["parent"], d)
    T = s["tokens"].shape[1]
    for b, (way, n, t) in enumerate(want):
        got = (path[b].tolist(), int(count[b]), int(token[b]))
        assert got == (way + [-1] * (T - n), n, t), (b, got, want[b])
    return want


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 2, 5), (5, 5, 1000), (7, 17, 1024), (3, 33, 1025), (2, 70, 4999), (4, 9, 40000)])
def test_verify(dtype, draft, tree, B, T, V):
    check(problem(B, T, V, dtype, draft, tree, seed=B + T))


@pytest.mark.parametrize("draft", [True, False])
def test_verify_ragged_and_one_tree(draft):
    s = problem(6, 20, 300, draft=draft, tree=True, seed=3)
    check(s, [20, 0, 1, 2, -4, 99])
    s["parent"] = s["parent"][0]
    check(s, [20, 19, 1, 20, 7, 20])


def test_every_child_is_rejected_and_tried_in_order():
    """Children of the root alone, far from the target: sums for each of them, one after the other."""
    g = torch.Generator().manual_seed(1)
    s = problem(40, 12, 2500, near=4.0, seed=5)
    s["parent"] = torch.tensor([-1] + [0] * 11, dtype=I32)
    for b in range(40):
        s["tokens"][b, 1:] = torch.multinomial(s["draft"][b, 0], 11, replacement=True, generator=g).int()
    found = check(s)
    assert {n for _, n, _ in found} == {1, 2} and len({way[1] for way, n, _ in found if n == 2}) > 3
    s["draft"] = None
    check(s)


@pytest.mark.parametrize("B,near", [(3, 0.6), (4, 4.0), (9, 1.5), (32, 2.0)])
def test_long_rows_of_some_trees(B, near):
    """Sums made by launches of their own, as many as walks ask for and fewer."""
    s = problem(B, 14, 66000, near=near, tree=True, seed=B)
    drafted = [14] * B
    drafted[0], drafted[1], drafted[-1] = 0, 2, 13
    found = check(s, drafted)
    assert len({n for _, n, _ in found}) > 1
    s["draft"] = s["target"].clone()           # nothing is ever left
    s["target"] = s["target"] * 0.5
    s["uniform"][:, 1:] = 0.75
    check(s)


@pytest.mark.parametrize("tree", [False, True])
def test_equal_probabilities_accept_all(tree):
    s = problem(3, 9, 700, tree=tree, seed=2, near=0.0)
    s["draft"] = s["target"]
    s["uniform"][:, 1:] = 1 - 2.0 ** -24
    for way, n, _ in check(s):
        assert tree or n == 9


def test_nothing_left():
    """A drafted token that no probability speaks for, and p below q wherever it is not zero."""
    p = torch.zeros(4, 3, 50)
    p[:, :, 7], p[0, :, 9] = 0.5, 0.5
    q = torch.zeros(4, 3, 50)
    q[:, :, 7], q[:, :, 3] = 0.75, 0.25
    p[2] = 0.0
    tokens = torch.tensor([[0, 3, 7], [0, 3, 3], [0, 7, 7], [0, 7, 3]], dtype=I32)
    u = torch.full((4, 3), 0.9)
    s = dict(tokens=tokens, target=p, uniform=u, draft=q, parent=None)
    found = check(s)
    assert found[2][2] == -1 and found[1][2] == 7
    s["draft"] = None
    check(s)
    s["parent"] = torch.tensor([-1, 0, 0], dtype=I32)
    check(s)
    s["draft"] = q
    check(s)


def test_probabilities_that_are_none():
    """NaN, infinite and negative ones count as zero; tokens and parents outside are passed over."""
    for draft in (True, False):
        s = problem(5, 8, 200, draft=draft, tree=True, seed=8)
        s["target"][:, 0, ::3] = math.nan
        s["target"][:, 1, 5], s["target"][:, 2, ::2] = math.inf, -1.0
        if draft:
            s["draft"][:, 0, 1::3] = math.nan
        s["tokens"][0, 2], s["tokens"][1, 1], s["tokens"][2, 3] = -1, 200, 10 ** 9
        s["parent"][3, 2], s["parent"][3, 4], s["parent"][4, 1] = 5, -3, 1
        check(s)


def test_a_token_twice_among_chosen_ones():
    """The second one is never accepted, whatever the random number."""
    p = torch.softmax(torch.randn(8, 6, 12, generator=torch.Generator().manual_seed(2)), -1)
    tokens = torch.tensor([[0, 4, 4, 5, 4, 5]] * 8, dtype=I32)
    u = torch.rand(8, 6, generator=torch.Generator().manual_seed(3))
    u[:, 1], u[:, 2] = 0.99999, 0.0
    u[4:, 3], u[4:, 4:] = 0.99999, 0.0
    check(dict(tokens=tokens, target=p, uniform=u, draft=None, parent=torch.tensor([-1, 0, 0, 0, 0, 0], dtype=I32)))


def test_random_numbers_at_the_ends():
    for value in (0.0, 1 - 2.0 ** -24, 0.5):
        for draft in (True, False):
            s = problem(4, 6, 3000, draft=draft, tree=True, seed=4)
            s["uniform"].fill_(value)
            s["target"][:, :, :1500] = 0.0
            check(s)


def test_distribution():
    """Tokens behind the root follow the target's probabilities, drawn or chosen, whatever was drafted: 60000 sequences, within five deviations."""
    N, V = 60000, 6
    g = torch.Generator().manual_seed(0)
    p, q = (torch.softmax(torch.randn(4, V, generator=g), -1) for _ in range(2))
    for draft in (True, False):
        tokens = torch.zeros(N, 4, dtype=I32)
        tokens[:, 1:] = torch.multinomial(q[0], 3 * N, replacement=True, generator=g).view(N, 3).int() if draft else torch.topk(q[0], 3).indices.int()
        u = torch.rand(N, 4, generator=g)
        path, count, token = kv.verify(put(tokens), put(p).expand(N, 4, V), put(u), draft=put(q).expand(N, 4, V) if draft else None,
                                       parent=torch.tensor([-1, 0, 0, 0], dtype=I32, device=DEV))
        path, count, token = path.cpu(), count.cpu(), token.cpu()
        first = torch.where(count > 1, tokens[torch.arange(N), path[:, 1].clamp(min=0).long()], token)
        share = torch.bincount(first.long(), minlength=V) / N
        assert ((share - p[0]).abs() < 5 * (p[0] * (1 - p[0]) / N).sqrt()).all()


def test_verify_views_and_large_vocabularies():
    """Rows off 16 bytes, strides between nodes and sequences, and a vocabulary of many segments."""
    s = problem(3, 4, 200003, seed=6)
    wide = torch.zeros(3, 5, 200010, device=DEV)
    wide[:, :4, 3:200006] = put(s["target"])
    want = check(s)
    t = wide[:, :4, 3:200006]
    u = torch.zeros(3, 9, device=DEV)
    u[:, 2:6] = put(s["uniform"])
    path, count, token = kv.verify(put(s["tokens"]), t, u[:, 2:6], draft=put(s["draft"]).transpose(0, 1).contiguous().transpose(0, 1))
    assert [(int(c), int(x)) for c, x in zip(count, token)] == [(n, x) for _, n, x in want]
    s = problem(1, 3, 5, seed=6)
    check(s, ws=torch.empty(kv.verify_workspace_bytes(1, 3, 5), dtype=torch.uint8, device=DEV))


def test_the_most_nodes():
    check(problem(2, 1024, 60, draft=False, tree=True, seed=1, wide=2))
    check(problem(2, 1024, 60, draft=True, tree=True, seed=2, wide=4, near=0.1))
    s = problem(2, 1024, 40, draft=False, seed=3)
    s["parent"] = torch.tensor([-1] + [0] * 1023, dtype=I32)       # 1023 children, of 40 tokens
    s["uniform"][:, 1:] = 1 - 2.0 ** -24
    check(s)


def test_verify_in_graphs_at_once():
    problems = [problem(8, 6, 5000, tree=True, seed=s) for s in (1, 2)]
    on = [{k: put(v) for k, v in s.items()} for s in problems]
    want = [kv.verify(s["tokens"], s["target"], s["uniform"], draft=s["draft"], parent=s["parent"]) for s in on]
    graphs, got = [], []
    torch.cuda.synchronize()
    for s in on:
        g = torch.cuda.CUDAGraph()
        ws = torch.empty(kv.verify_workspace_bytes(8, 6, 5000), dtype=torch.uint8, device=DEV)
        with torch.cuda.graph(g):
            r = kv.verify(s["tokens"], s["target"], s["uniform"], draft=s["draft"], parent=s["parent"], ws=ws)
        graphs.append((g, ws))
        got.append(r)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for r in got:
            for t in r:
                t.fill_(77)
        torch.cuda.synchronize()
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for r, w in zip(got, want) for a, b in zip(r, w))


# ----------------------------------------------------------------- accept --
def rows(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 72), (torch.float8_e5m2, 64), (BF16, 8), (torch.float8_e5m2, 8), (BF16, 256)])
@pytest.mark.parametrize("layout", ["shd", "hsd", "paged16", "paged64"])
@pytest.mark.parametrize("T", [1, 7, 64, 150])
def test_accept(dtype, D, layout, T):
    B, H, S = 4, 3, 200
    page = int(layout[5:]) if layout.startswith("paged") else 0
    per = -(-S // page) if page else 0
    first, second = (B * per + 1, page) if page else (B, S)
    k, v = rows((first, second, H, D), dtype, 1), rows((first, second, H, D), dtype, 2)
    table = torch.randperm(first, generator=torch.Generator().manual_seed(3))[:B * per].view(B, per).to(I32) if page else None
    if page:
        table[2, 2] = -1
    rng = random.Random(T)
    path = torch.full((B, T), -1, dtype=I32)
    count = []
    for b in range(B):
        way = sorted(rng.sample(range(1, T), rng.randint(0, T - 1))) if T > 1 else []
        path[b, :len(way) + 1] = torch.tensor([0] + way, dtype=I32)
        count.append(len(way) + 1)
    count[1] = 0 if T == 7 else count[1]
    length = [0, 33, 45, S - 20]
    want = [t.clone() for t in (k, v)]
    for t, w in zip((k, v), want):
        for b in range(B):
            for j in range(count[b]):
                src, dst = step.place(t, table, b, length[b] + int(path[b, j])), step.place(t, table, b, length[b] + j)
                if src is not None and dst is not None and path[b, j] > j:
                    w[dst] = t[src]
    turn = (lambda t: t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)) if layout == "hsd" else put  # noqa: E731
    dk, dv = turn(k), turn(v)
    assert kv.accept(dk, dv, torch.tensor(length, dtype=I32, device=DEV), put(path), torch.tensor(count, dtype=I32, device=DEV), table=put(table)) is None
    for got, w in zip((dk, dv), want):
        assert torch.equal(bits(got.cpu()), bits(w))


def test_paths_that_are_none():
    """Entries outside, numbers that do not grow, counts outside: in bounds, and rows behind the drafted ones left as they were."""
    k, v = rows((3, 64, 2, 64), BF16, 1), rows((3, 64, 2, 64), BF16, 2)
    path = torch.tensor([[5, -9, 2 ** 30, 3], [0, 0, 0, 0], [3, 2, 1, 0]], dtype=I32)
    dk, dv = put(k), put(v)
    kv.accept(dk, dv, torch.tensor([-2 ** 31, 63, 2 ** 31 - 1], dtype=I32, device=DEV), put(path), torch.tensor([2 ** 30, 4, -1], dtype=I32, device=DEV))
    assert torch.equal(dk.cpu(), k) and torch.equal(dv.cpu(), v)
    kv.accept(dk, dv, torch.tensor([0, 10, 60], dtype=I32, device=DEV), put(path), torch.tensor([9, 4, 4], dtype=I32, device=DEV))
    assert torch.equal(dk.cpu()[:, 4:60], k[:, 4:60])


# ------------------------------------------------------------------ pages --
def tables(S, E, page, pages, seed, share=True, absent=0.0):
    """Tables whose rows share prefixes, with entries behind the tokens that are not to be looked at."""
    rng = random.Random(seed)
    free = list(range(pages))
    rng.shuffle(free)
    table, length = [], []
    for s in range(S):
        if s and share and rng.random() < 0.6:
            other = rng.randrange(s)
            n = rng.randint(0, length[other]) if rng.random() < 0.5 else length[other]
            row = list(table[other])
        else:
            n = rng.randint(0, E * page)
            n = n // page * page if rng.random() < 0.2 else n
            row = []
            while len(row) < -(-n // page) and free:
                row.append(free.pop())
            n = min(n, len(row) * page)
            row += [rng.choice([-1, rng.randrange(pages), 2 ** 30]) for _ in range(E - len(row))]
        row = [-1 if rng.random() < absent else x for x in row]
        table.append(row)
        length.append(n)
    return torch.tensor(table, dtype=I32), torch.tensor(length, dtype=I32)


def check_fork(table, length, parent, pages, page, room=0, held=None):
    t, n, moves, left = kv.fork(put(table), put(length), put(parent), pages, page, room=room, held=put(held))
    want = step.fork(table, length, parent, pages, page, room, held)
    assert t.tolist() == want[0]
    assert (n.tolist(), moves.tolist(), int(left)) == (want[1], want[2], want[3])
    return t, n, moves, left


@pytest.mark.parametrize("S,B,E,page,pages", [(1, 1, 1, 16, 1), (1, 5, 3, 16, 20), (4, 4, 7, 32, 100), (9, 30, 5, 16, 60), (40, 60, 300, 16, 9000),
                                              (3, 1100, 4, 64, 3000), (64, 64, 40, 16, 20000), (5, 5, 600, 16, 70000)])
@pytest.mark.parametrize("room", [0, 1, 40])
@pytest.mark.parametrize("absent", [0.0, 0.1])
def test_fork(S, B, E, page, pages, room, absent):
    """Continued, forked and dropped sequences, also with fewer free pages than they need."""
    table, length = tables(S, E, page, pages, S + B + E, absent=absent)
    rng = random.Random(B)
    parent = torch.tensor([rng.choice([-1, S, 10 ** 6]) if rng.random() < 0.1 else rng.randrange(S) for _ in range(B)], dtype=I32)
    check_fork(table, length, parent, pages, page, room)
    held = torch.rand(pages, generator=torch.Generator().manual_seed(1)) < 0.3
    check_fork(table, length, parent, pages, page, room, held)
    check_fork(table, length, torch.full((B,), -1, dtype=I32), pages, page, room, held)


def test_fork_lengths_outside():
    table, _ = tables(5, 6, 16, 40, 2)
    for length in ([-1, 0, 96, 97, 2 ** 31 - 1], [16, 17, 95, 80, -2 ** 31]):
        check_fork(table, torch.tensor(length, dtype=I32), torch.tensor([0, 1, 2, 3, 4, 4, 3, 2], dtype=I32), 40, 16, 20)
    everything = torch.zeros(40, dtype=torch.bool)
    everything[:] = True
    check_fork(table, torch.tensor([10, 20, 30, 40, 50], dtype=I32), torch.tensor([0, 1, 2, 3, 4], dtype=I32), 40, 16, 20, everything)


def test_a_last_page_that_is_whole_for_another():
    """A sequence cut inside a page that another has whole gets a copy, and so do all but the first of those that fill one on."""
    table = torch.tensor([[3, 4, 5, -1], [3, 4, 5, -1], [7, -1, -1, -1]], dtype=I32)
    t, n, moves, left = check_fork(table, torch.tensor([40, 24, 9], dtype=I32), torch.tensor([0, 1, 0, 2, 2], dtype=I32), 10, 16)
    assert moves.tolist() == [[-1, -1], [4, 0], [5, 1], [-1, -1], [7, 2]] and int(left) == 3
    assert t.tolist() == [[3, 4, 5, -1], [3, 0, -1, -1], [3, 4, 1, -1], [7, -1, -1, -1], [2, -1, -1, -1]]


@pytest.mark.parametrize("S,E,page,pages", [(1, 1, 16, 1), (3, 4, 16, 30), (20, 50, 16, 2000), (70, 30, 32, 9000), (9, 900, 16, 70000)])
def test_compact(S, E, page, pages):
    table, length = tables(S, E, page, pages, S + E, absent=0.02)
    held = torch.rand(pages, generator=torch.Generator().manual_seed(1)) < 0.1
    for h in (None, held):
        t, moves, used = kv.compact(put(table), put(length), pages, page, held=put(h))
        want = step.compact(table, length, pages, page, h)
        assert (t.tolist(), int(used)) == (want[0], want[2])
        assert moves.shape[0] == min(S * E, pages // 2)
        assert moves.tolist() == want[1] + [[-1, -1]] * (moves.shape[0] - len(want[1]))


def pools(pages, page):
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return [r(pages, page, 3, 72).to(BF16), r(pages, 3, page, 64).to(F16).transpose(1, 2), (r(pages, page, 2, 40) * 30).to(torch.int8), r(pages, page // 16, 3),
            r(pages, page, 5, 128).to(BF16)[:, :, 1:4], r(pages, page, 8, 64).to(BF16)[:, :, 2:4, :32], (r(pages, page, 3, 7) * 9).to(torch.int8)[:, :, :, 1:4]]


def test_copy_pages():
    """Keys, values and scales of any type and strides in one call; pages outside are passed over, all others left as they were."""
    moves = torch.tensor([[0, 9], [-1, -1], [5, 7], [3, 12], [12, 3], [2 ** 30, 1], [5, 8], [11, 4], [1, -5]], dtype=I32)
    for count in (1, 4, 7):
        t = pools(12, 32)[:count]
        want = [x.clone() for x in t]
        for w, x in zip(want, t):
            for a, b in moves.tolist():
                if 0 <= a < 12 and 0 <= b < 12:
                    w[b] = x[a]
        kv.copy_pages(put(moves), *t)
        assert all(torch.equal(a, b) for a, b in zip(t, want))
    t = pools(12, 32)
    for x in t:                             # each alone: the unit of copying is its own
        w = x.clone()
        w[7] = x[5]
        kv.copy_pages(torch.tensor([[5, 7]], dtype=I32, device=DEV), x)
        assert torch.equal(x, w)
    kv.copy_pages(torch.empty(0, 2, dtype=I32, device=DEV), t[0])


def test_copy_pages_past_32_bits():
    pool = torch.zeros(2500, 1024, 8, 128, dtype=torch.int16, device=DEV)
    pool[2] = torch.randint(-2 ** 15, 2 ** 15, (1024, 8, 128), device=DEV, dtype=torch.int16)
    kv.copy_pages(torch.tensor([[2, 2499]], dtype=I32, device=DEV), pool)
    assert torch.equal(pool[2499], pool[2]) and not pool[2498].any()


def contents(pool, table, length, page):
    """Each sequence's tokens."""
    return [torch.cat([pool[p] for p in row[:-(-n // page)]])[:n] if n else pool[0][:0] for row, n in zip(table.tolist(), length.tolist())]


def test_sequences_keep_their_tokens():
    """Forked, filled on, dropped and compacted, over and over: each sequence reads as if it had a cache of its own."""
    page, pages, E, H, D = 16, 120, 8, 2, 64
    pool = torch.randn(pages, page, H, D, device=DEV).to(BF16)
    other = torch.randn(pages, page, H, D, device=DEV).to(BF16)
    rng = random.Random(7)
    table = torch.full((3, E), -1, dtype=I32, device=DEV)
    length = torch.zeros(3, dtype=I32, device=DEV)
    mine = [torch.empty(0, H, D, dtype=BF16, device=DEV) for _ in range(3)]
    for it in range(25):
        parent = [rng.randrange(len(mine)) if rng.random() < 0.9 else -1 for _ in range(rng.randint(1, 6))]
        T = rng.randint(1, 20)
        mine = [mine[p] if p >= 0 and len(mine[p]) + T <= E * page else None for p in parent]
        parent = [p if m is not None else -1 for p, m in zip(parent, mine)]
        table, length, moves, left = kv.fork(table, length, torch.tensor(parent, dtype=I32, device=DEV), pages, page, room=T)
        kv.copy_pages(moves, pool, other)
        assert int(left) >= 0
        if it % 3 == 2:
            table, moves, used = kv.compact(table, length, pages, page)
            kv.copy_pages(moves, pool, other)
            assert int(used) <= pages and int(table.max()) < int(used)
            # the room was not in use: it is given again
            table, length, moves, left = kv.fork(table, length, torch.arange(len(parent), dtype=I32, device=DEV), pages, page, room=T)
            kv.copy_pages(moves, pool, other)
            assert not (moves >= 0).any()
        new = torch.randn(len(parent), T, H, D, device=DEV).to(BF16)
        drafted = torch.tensor([T if m is not None else 0 for m in mine], dtype=I32, device=DEV)
        kv.append(None, new, -new, pool, other, length, table=table, drafted=drafted)
        length = length + drafted
        mine = [torch.cat((m, new[b])) if m is not None else new[b][:0] for b, m in enumerate(mine)]
        for a, b, c in zip(contents(pool, table, length, page), contents(other, table, length, page), mine):
            assert torch.equal(a, c) and torch.equal(b, -c)


def test_a_step_of_drafted_trees():
    """Append, attend, verify, accept and fork as a server runs them: the cache then is that of the accepted tokens alone, and attention over it is a chain's."""
    B, T, hq, H, D, page, V = 3, 12, 8, 2, 64, 16, 500
    pages, E = 60, 10
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    k, v = r(pages, page, H, D).to(BF16), r(pages, page, H, D).to(BF16)
    length = torch.tensor([40, 0, 63], dtype=I32, device=DEV)
    table = torch.full((B, E), -1, dtype=I32, device=DEV)
    table[0, :3], table[2, :4] = torch.tensor([50, 7, 9], dtype=I32, device=DEV), torch.tensor([1, 2, 3, 4], dtype=I32, device=DEV)
    table, length, moves, _ = kv.fork(table, length, torch.arange(B, dtype=I32, device=DEV), pages, page, room=T)
    s = {x: put(y) for x, y in problem(B, T, V, tree=True, seed=9).items()}
    parent = s["parent"].cpu()
    tree = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            at = i
            while at >= 0:
                tree[b, i, at] = True
                at = int(parent[b, at])
    q, nk, nv = r(B, T, hq, D).to(BF16), r(B, T, H, D).to(BF16), r(B, T, H, D).to(BF16)
    kv.append(None, nk, nv, k, v, length, table=table)
    out = kv.attend(q, k, v, length, table=table, tree=put(tree))
    path, count, token = kv.verify(s["tokens"], s["target"], s["uniform"], draft=s["draft"], parent=s["parent"])
    kv.accept(k, v, length, path, count, table=table)
    assert int(count.max()) > 1
    for b in range(B):
        n, m = int(length[b]), int(count[b])
        way = path[b, :m].long()
        rows_k = contents(k, table[b:b + 1], length[b:b + 1] + m, page)[0]
        assert torch.equal(rows_k[n:], nk[b, way])
        chain = kv.attend(q[b:b + 1, way], k, v, length[b:b + 1], table=table[b:b + 1])
        assert torch.allclose(chain[0].float(), out[b, way].float(), atol=2.0 ** -6, rtol=2.0 ** -6)
    assert (token >= 0).all()


def test_pages_and_accepted_tokens_in_a_graph_and_on_another_stream():
    """A step's bookkeeping captured and replayed with other tables in the same memory, and on a stream of its own."""
    page, pages, E, S, B, T = 16, 400, 9, 20, 30, 12
    pool = torch.randn(pages, page, 2, 64, device=DEV).to(BF16)
    other = torch.randn(pages, page, 2, 64, device=DEV).to(BF16)
    sets = []
    for seed in (1, 2):
        table, length = tables(S, E, page, pages, seed)
        rng = random.Random(seed)
        parent = torch.tensor([rng.randrange(-1, S) for _ in range(B)], dtype=I32)
        path = torch.tensor([[0] + sorted(rng.sample(range(1, T), 5)) + [-1] * (T - 6) for _ in range(B)], dtype=I32)
        sets.append([put(x) for x in (table, length, parent, path, torch.randint(0, 7, (B,), generator=torch.Generator().manual_seed(seed)).to(I32))])
    mine = [x.clone() for x in sets[0]]
    a, b = pool.clone(), other.clone()
    ws = torch.empty(kv.pages_workspace_bytes(pages, B, E), dtype=torch.uint8, device=DEV)

    def run(k, v, table, length, parent, path, count, stream=None):
        t, n, moves, left = kv.fork(table, length, parent, pages, page, room=T, ws=ws, stream=stream)
        kv.copy_pages(moves, k, v, stream=stream)
        kv.accept(k, v, n, path, count, table=t, stream=stream)
        c, moved, used = kv.compact(t, n, pages, page, stream=stream)
        kv.copy_pages(moved, k, v, stream=stream)
        return t, n, moves, left, c, moved, used

    want = []
    for s in sets:
        k, v = pool.clone(), other.clone()
        want.append([x.clone() for x in (*run(k, v, *s), k, v)])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    k, v = pool.clone(), other.clone()
    torch.cuda.synchronize()
    got = run(k, v, *sets[0], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*got, k, v), want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(a, b, *mine)
    for i in (0, 1, 0, 1):
        for x, y in zip(mine, sets[i]):
            x.copy_(y)
        a.copy_(pool), b.copy_(other)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*got, a, b), want[i]))
