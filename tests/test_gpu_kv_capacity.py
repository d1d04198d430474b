"""kv.attend where length + drafted passes the cache's capacity: the drafted
tokens behind its end are not there, whatever a tree names."""
import math

import pytest
import torch

import kv_reference as ref
from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV, E5M2, F16, bits, check, large, make, put, tree_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout,cache", [("shd", BF16), ("hsd", F16), ("shd", E5M2), ("paged16", BF16)])
@pytest.mark.parametrize("cap", [3, 50, 79, 97, 400])
@pytest.mark.parametrize("T,hq,H,D", [(3, 4, 2, 64), (5, 6, 1, 128), (20, 6, 2, 72), (9, 2, 2, 256)])
def test_trees_past_the_end(layout, cache, cap, T, hq, H, D):
    """From one token inside to none; a whole tree, the tokens behind the end
    alone, and any mask."""
    q, k, v, table = make(5, T, hq, H, D, cap, F16 if cache == F16 else BF16, cache, layout, seed=cap + T)
    held = cap if table is None else table.shape[1] * k.shape[1]
    length = [max(held - x, 0) for x in (1, 0, 2, T, T - 1)]
    whole = torch.ones(T, T, dtype=torch.bool)
    lone = torch.zeros(T, T, dtype=torch.bool)
    lone[:, -1] = True
    for tree in (whole, lone, tree_of(T, cap, 5)):
        check(q, k, v, length, table=table, tree=tree, layout=layout)
        check(q, k, v, length, table=table, tree=tree, drafted=[T, T, T - 1, 1, 2], layout=layout)


def test_an_empty_cache_row_behind_the_end():
    """Nothing cached that is seen and nothing drafted that is there: zeros and -inf."""
    q, k, v, table = make(1, 3, 2, 1, 64, 48, layout="paged16", seed=1)
    table[:] = -1
    out, lse, _ = check(q, k, v, [48], table=table, tree=torch.ones(3, 3, dtype=torch.bool))
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("B,T,hq,H,D,S,cache,layout", [(5, 70, 32, 8, 128, 2413, BF16, "shd"), (5, 70, 32, 8, 64, 2405, E5M2, "hsd"),
                                                       (5, 24, 96, 32, 72, 1763, F16, "hsd")])
def test_trees_past_the_end_of_shared_keys(B, T, hq, H, D, S, cache, layout):
    q, k, v, _ = large(B, T, hq, H, D, S, cache, layout, S)
    g = torch.Generator().manual_seed(S)
    G = hq // H
    length = torch.tensor([S - 1, S, S - T + 1, S - T - 1, S - 2], dtype=torch.int32)
    drafted = torch.tensor([T, T, T, T, 3], dtype=torch.int32)
    for b in range(B):                            # memory behind the tokens that are there
        end = min(S, int(length[b]) + int(drafted[b]))
        for t in (k, v):
            bits(t)[b, end:] = bits(torch.full((1,), math.nan).to(cache)).to(DEV)
    tree = torch.rand(B, T, T, generator=g) < 0.5
    tree[0] = True
    w, lse = torch.zeros(B, H, S, device=DEV), torch.full((B, T, hq), 3.0, device=DEV)
    out = kv.attend(q, k, v, length.to(DEV), tree=put(tree), drafted=drafted.to(DEV), score=w, lse=lse)
    for b, h in ((0, 0), (1, H - 1), (2, 1), (3, 2), (4, H // 2)):
        at, heads = slice(b, b + 1), slice(h * G, h * G + G)
        want = ref.attend(q[at, :, heads].cpu(), k[at, :, h:h + 1].cpu(), v[at, :, h:h + 1].cpu(), length[at], tree=tree[at], drafted=drafted[at])
        ref.within(out[at, :, heads], want["out"], want["out_bound"], f"out {b} {h}")
        ref.within(lse[at, :, heads], want["lse"], want["lse_bound"], f"lse {b} {h}")
        ref.within(w[at, h:h + 1], want["weight"], want["weight_bound"], f"score {b} {h}")
