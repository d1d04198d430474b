"""kv.evict against sorting, and the operators' whole run: append, attend with
weights, evict, encode, decode, attend again."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref
import oracle
from lossless_bf16_tensor_amd import kv, uzip

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, E5M2 = torch.bfloat16, torch.float16, torch.float8_e5m2


def bits(t):
    return t.view(torch.uint8) if t.dtype == E5M2 else t.view(torch.int16)


def scores(kind, B, H, S, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.exp(2 * torch.randn(B, H, S, generator=g))
    if kind == "ties":
        x = torch.randint(0, 4, (B, H, S), generator=g).float()
    elif kind == "equal":
        x = torch.full((B, H, S), 0.5)
    elif kind == "signed":
        x = torch.randn(B, H, S, generator=g)
        x[..., ::5] = 0.0
        x[..., 1::5] = -0.0
    elif kind == "odd":
        x[..., ::7] = math.nan
        x[..., 1::7] = math.inf
        x[..., 2::7] = -math.inf
        x[..., 3::7] = 2.0 ** -149
    return x


def run(B, H, S, D, lens, keep, sink, recent, kind="plain", cache=BF16, layout="shd", seed=0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(cache)  # noqa: E731
    table = None
    if layout.startswith("paged"):
        page = int(layout[5:])
        per = -(-S // page)
        k, v = mk(B * per + 1, page, H, D), mk(B * per + 1, page, H, D)
        table = torch.randperm(B * per + 1, generator=g)[:B * per].view(B, per).to(torch.int32)
    else:
        k, v = mk(B, S, H, D), mk(B, S, H, D)
    score = scores(kind, B, H, S, seed)
    n = torch.tensor(lens, dtype=torch.int32)
    kept = ref.evict(score, n, keep, sink, recent, S)
    put = (lambda t: bits(t).transpose(1, 2).contiguous().to(DEV).transpose(1, 2).view(cache)) if layout == "hsd" else (lambda t: t.to(DEV))
    gk, gv, gs, gn, gi = kv.evict(put(k), put(v), score.to(DEV), n.to(DEV), keep, sink=sink, recent=recent,
                                  table=None if table is None else table.to(DEV))
    gk, gv, gs, gn, gi = (t.cpu() for t in (bits(gk), bits(gv), gs, gn, gi))
    for b in range(B):
        assert int(gn[b]) == len(kept[b][0])
        for h in range(H):
            at = torch.tensor(kept[b][h], dtype=torch.int64)
            m = at.numel()
            assert gi[b, h, :m].tolist() == at.tolist(), (b, h)
            assert (gi[b, h, m:] == -1).all() and not gk[b, m:, h].any() and not gv[b, m:, h].any() and not gs[b, h, m:].any()
            want = (bits(t)[b, at, h] if table is None else bits(t)[table[b, at // k.shape[1]].long(), at % k.shape[1], h] for t in (k, v))
            for got, w in zip((gk, gv), want):
                assert torch.equal(got[b, :m, h], w)
            assert torch.equal(gs[b, h, :m].view(torch.int32), score[b, h, at].view(torch.int32))


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signed", "odd"])
@pytest.mark.parametrize("S,keep,sink,recent", [(1, 1, 0, 0), (64, 7, 2, 3), (65, 65, 4, 4), (300, 299, 0, 1), (300, 8, 8, 0),
                                                (300, 8, 3, 5), (2049, 500, 4, 64), (5000, 1, 0, 0)])
def test_choice(kind, S, keep, sink, recent):
    run(2, 3, S, 8, [S, max(0, S - 9)], keep, sink, recent, kind, seed=S)


@pytest.mark.parametrize("cache", [BF16, F16, E5M2])
@pytest.mark.parametrize("layout", ["shd", "hsd", "paged16", "paged64"])
@pytest.mark.parametrize("D", [8, 72, 128, 256])
def test_copies(cache, layout, D):
    run(5, 3, 200, D, [200, 0, 1, 33, 90], 33, 1, 9, "plain", cache, layout, seed=D)


@pytest.mark.parametrize("S,keep,sink,recent", [(4096, 1000, 0, 0), (4097, 4000, 7, 100), (16385, 16384, 1, 0), (32768, 20000, 0, 9),
                                                (32769, 17, 17, 0), (40000, 30, 10, 20), (40960, 40959, 0, 0), (50000, 25000, 9000, 10000)])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
def test_lengths_at_the_edges_of_what_a_workgroup_holds(S, keep, sink, recent, kind):
    run(1, 2, S, 8, [S], keep, sink, recent, kind, seed=S)
    run(2, 1, S, 8, [S - 3, keep + 1], keep, sink, recent, kind, seed=S + 1)


def test_long_rows():
    run(1, 2, 70001, 8, [70001], 20011, 3, 1000, "ties", seed=1)
    run(2, 1, 131072, 8, [131072, 100000], 13000, 0, 0, "plain", seed=2)
    run(1, 1, 131072, 8, [131072], 131071, 0, 0, "odd", seed=3)


def test_lengths_outside_the_cache_and_absent_pages():
    run(3, 2, 100, 16, [-4, 101, 2 ** 31 - 1], 40, 2, 2)
    k = torch.ones(4, 16, 2, 64, dtype=BF16, device=DEV)
    table = torch.tensor([[0, -1, 9]], dtype=torch.int32, device=DEV)
    score = torch.arange(96, dtype=torch.float32, device=DEV).view(1, 2, 48)
    gk, gv, _, gn, gi = kv.evict(k, k, score, torch.tensor([48], dtype=torch.int32, device=DEV), 20, sink=4, table=table)
    assert gi[0, 0].tolist() == [0, 1, 2, 3] + list(range(32, 48)) and int(gn) == 20
    assert (gk[0, :4] == 1).all() and not gk[0, 4:].any() and not gv[0, 4:].any()


def test_scores_are_float32_whatever_the_default_type():
    default = torch.get_default_dtype()
    try:
        for t in (BF16, torch.float64):
            torch.set_default_dtype(t)
            k = torch.ones(1, 40, 2, 64, dtype=BF16, device=DEV)
            score = torch.rand(1, 2, 40, dtype=torch.float32).to(DEV)
            kept = kv.evict(k, k, score, torch.tensor([40], dtype=torch.int32, device=DEV), 40)[2]
            assert kept.dtype == torch.float32 and torch.equal(kept, score)
    finally:
        torch.set_default_dtype(default)


def test_two_long_cuts_at_once():
    """On two streams, each with a workspace of its own."""
    B, H, S, keep = 2, 2, 60000, 9000
    g = torch.Generator().manual_seed(5)
    k = torch.randn(B, S, H, 16, generator=g).to(BF16).to(DEV)
    score = [scores(kind, B, H, S, 6).to(DEV) for kind in ("plain", "ties")]
    n = torch.tensor([S, 50001], dtype=torch.int32, device=DEV)
    want = [kv.evict(k, k, x, n, keep, sink=2, recent=40) for x in score]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[kv.evict(k, k, x, n, keep, sink=2, recent=40, stream=s) for x, s in zip(score, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_same_choice_every_time_and_in_a_graph():
    B, H, S, D, keep = 2, 4, 9000, 64, 1000
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(B, S, H, D, generator=g).to(BF16).to(DEV) for _ in range(2))
    score = scores("ties", B, H, S, 4).to(DEV)
    n = torch.tensor([S, 5000], dtype=torch.int32, device=DEV)
    ws = torch.empty(kv.evict_workspace_bytes(B, H, S), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.evict(k, v, score, n, keep, recent=10, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kv.evict(k, v, score, n, keep, recent=10, ws=ws)
    for seed in range(4):
        score.copy_(scores("ties" if seed % 2 else "plain", B, H, S, seed))
        n.copy_(torch.tensor([S - seed, 5000 - 2000 * seed], dtype=torch.int32).clamp(min=0))
        ws.fill_(seed * 50)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = kv.evict(k, v, score, n, keep, recent=10)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_operators_run_together():
    """A prompt appended, its last tokens' weights gathered, the cache cut,
    encoded, decoded as the receiver would, and a drafted tree attended over
    it: equal, bit for bit, to attending over the kept tokens themselves."""
    B, S, H, G, D, keep, T = 2, 700, 2, 4, 128, 256, 6
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g).to(BF16).to(DEV)  # noqa: E731
    kc, vc = (torch.zeros(B, S, H, D, dtype=BF16, device=DEV) for _ in range(2))
    freq = kv.rope_freq(D).to(DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    prompt = torch.tensor([700, 412], dtype=torch.int32, device=DEV)
    q = kv.append(mk(B, S, H * G, D), mk(B, S, H, D), mk(B, S, H, D), kc, vc, zero, freq, drafted=prompt)

    window = 32
    score = torch.zeros(B, H, S, device=DEV)
    for b in range(B):                            # the last 32 prompt tokens observe the cache
        m = int(prompt[b])
        out = kv.attend(q[b:b + 1, m - window:m], kc[b:b + 1], vc[b:b + 1], prompt[b:b + 1] - window, score=score[b:b + 1])
        want = ref.attend(q[b:b + 1, m - window:m].cpu(), kc[b:b + 1].cpu(), vc[b:b + 1].cpu(), prompt[b:b + 1].cpu() - window)
        ref.within(out, want["out"], want["out_bound"])
        ref.within(score[b:b + 1], want["weight"], want["weight_bound"])
    room = keep + T
    k2, v2 = (torch.zeros(B, room, H, D, dtype=BF16, device=DEV) for _ in range(2))
    k1, v1, _, n1, index = kv.evict(kc, vc, score, prompt, keep, sink=4, recent=window)
    for b in range(B):
        for h in range(H):
            assert torch.equal(k1[b, :, h], kc[b, index[b, h].long(), h])

    for src, dst in ((k1, k2), (v1, v2)):         # the transfer
        words = src.view(torch.int16).reshape(-1)
        cb = uzip.calibrate(words)
        buf = uzip.encode(words, cb, 1024)
        total, _ = uzip.stream_bytes(buf)
        host = words.cpu().numpy().view(np.uint16)
        assert np.array_equal(buf[:total].cpu().numpy(), oracle.encode(host, 1024, np.array(cb.dec_list, np.uint8)))
        back = uzip.decode(buf[:total], cb, words.numel(), 1024).view(BF16).view_as(src)
        assert torch.equal(back.view(torch.int16), src.view(torch.int16))
        dst[:, :keep] = back

    tree = torch.tensor([[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [0, 0, 0, 1, 0, 0], [0, 0, 0, 1, 1, 0],
                         [1, 1, 0, 0, 0, 1]], dtype=torch.bool, device=DEV)
    pos = prompt[:, None] + (tree.sum(1).to(torch.int32) - 1)[None]     # depth in the tree behind the prompt
    new = [mk(B, T, h, D) for h in (H * G, H, H)]
    q2 = kv.append(*new, k2, v2, n1, freq, pos=pos)
    got = kv.attend(q2, k2, v2, n1, tree=tree)
    want = ref.attend(q2.cpu(), k2.cpu(), v2.cpu(), n1.cpu(), tree=tree.cpu())
    ref.within(got, want["out"], want["out_bound"])
    # the kept tokens gathered by hand, never encoded
    k3, v3 = k2.clone(), v2.clone()
    k3[:, :keep], v3[:, :keep] = k1, v1
    assert torch.equal(got, kv.attend(q2, k3, v3, n1, tree=tree))
