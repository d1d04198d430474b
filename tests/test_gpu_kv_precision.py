"""kv.attend where few bits would show: many small weights beside a large one,
queries whose elements lie far apart, weights rounded before their product."""
import math

import pytest
import torch

import kv_reference as ref
from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV, E5M2, F16, check, make, put, tree_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,cache", [(F16, F16), (BF16, BF16), (F16, E5M2), (BF16, E5M2)])
@pytest.mark.parametrize("B,T,hq,H,S,D", [(1, 1, 1, 1, 4096, 64), (2, 1, 24, 1, 3000, 256), (2048, 1, 1, 1, 4096, 128), (1, 65, 1, 1, 20000, 64),
                                          (128, 65, 8, 8, 4160, 64), (128, 65, 8, 8, 4160, 128)])
@pytest.mark.parametrize("at", [0, 2000])
def test_small_weights_beside_a_large_one(q, cache, B, T, hq, H, S, D, at):
    """One token's score is 18 above all others', as a first token's often is.
    Its values are zero, so the output is the others' share, N e^-18 / (1 + N
    e^-18) of their common value: a kernel that rounds weights of 2^-26 away
    loses them. Weights of FP16 products may be off by FP16's last step, 2^-24
    where the largest is 2^11, so by 2^-35 of it each; the sums of N weights in
    binary32 and the score's own rounding are far below the output's half step."""
    k, v = torch.zeros(1, S, 1, D), torch.full((1, S, 1, D), 1.5)
    k[:, at, :, 0], v[:, at] = 20.0, 0.0
    k, v = (t.to(cache).to(DEV).expand(B, S, H, D) for t in (k, v))
    x = torch.zeros(1, 1, 1, D)
    x[..., 0] = 1.0
    x = x.expand(B, T, hq, D).contiguous().to(q).to(DEV)
    n = torch.full((B,), S - T, dtype=torch.int32, device=DEV)
    seen = (S - T + 1 + torch.arange(T, dtype=torch.float64)).view(1, T, 1)       # a chain
    lse = torch.empty(B, T, hq, device=DEV)
    out = kv.attend(x, k, v, n, scale=0.9, lse=lse)
    small = (seen - 1) * math.exp(-18.0)
    want = (1.5 * small / (1 + small))[..., None].expand(B, T, hq, D)
    bound = want * (ref.HALF[q] + 2.0 ** -16) + 1.5 * S * 2.0 ** -35
    ref.within(out, want, bound, "out")
    ref.within(lse, (18.0 + torch.log1p(small)).expand(B, T, hq), torch.tensor(2.0 ** -17), "lse")


@pytest.mark.parametrize("T,hq,H,D", [(1, 4, 2, 128), (6, 8, 2, 64), (20, 6, 2, 72), (9, 8, 2, 256)])
@pytest.mark.parametrize("far", [20, 40, 100])
def test_queries_of_far_apart_elements(T, hq, H, D, far):
    """BF16 queries of an E5M2 cache with one element 2^far above the others,
    where the keys are zero, but for one where that still leaves the others a say."""
    q, k, v, _ = make(2, T, hq, H, D, 300, BF16, E5M2, seed=far + D)
    q[..., 3] = 2.0 ** far * torch.sign(q[..., 3])
    k = k.float()
    k[..., 3] = 0.0
    if far == 20:
        k[:, 7, :, 3] = 2.0 ** -14
    check(q, k.to(E5M2), v, [300 - T, 100])


def test_queries_of_far_apart_elements_share_keys():
    B, T, hq, H, D, S = 5, 70, 32, 8, 64, 2405
    g = torch.Generator().manual_seed(3)
    q = torch.randn(B, T, hq, D, generator=g)
    q[..., 5] *= 2.0 ** 30
    k, v = torch.randn(B, S, H, D, generator=g), torch.randn(B, S, H, D, generator=g).to(E5M2)
    k[..., 5] = 0.0
    q, k = q.to(BF16), k.to(E5M2)
    n = torch.tensor([S - T, 1000, 0, 2000, 1999], dtype=torch.int32)
    lse = torch.empty(B, T, hq, device=DEV)
    w = torch.zeros(B, H, S, device=DEV)
    out = kv.attend(q.to(DEV), k.to(DEV), v.to(DEV), n.to(DEV), lse=lse, score=w)
    for b, h in ((0, 0), (1, 7), (2, 3), (4, 5)):
        at, heads = slice(b, b + 1), slice(4 * h, 4 * h + 4)
        want = ref.attend(q[at, :, heads], k[at, :, h:h + 1], v[at, :, h:h + 1], n[at])
        ref.within(out[at, :, heads], want["out"], want["out_bound"], f"out {b} {h}")
        ref.within(lse[at, :, heads], want["lse"], want["lse_bound"], f"lse {b} {h}")
        ref.within(w[at, h:h + 1], want["weight"], want["weight_bound"], f"score {b} {h}")


@pytest.mark.parametrize("q,cache", [(BF16, BF16), (F16, F16), (F16, E5M2)])
@pytest.mark.parametrize("T,hq,H,D", [(1, 4, 2, 64), (3, 8, 2, 128), (30, 2, 2, 72), (9, 2, 2, 256)])
@pytest.mark.parametrize("n", [0, 3, 40, 1000])
def test_weights_are_not_rounded_to_the_caches_type(q, cache, T, hq, H, D, n):
    """Where the keys are not shared: weights in two terms, the first cut off, so
    that less than a step is left, and that rounded to half a step of itself:
    2^-7 2^-8 of the weight, or 2^-10 2^-11, or in FP16 its last step, 2^-35 of
    the largest. The rest is binary32. Scores are small, so that their own
    rounding is."""
    x, k, v, _ = make(2, T, hq, H, D, n + T, q, cache, seed=n + D, kscale=2.0 ** -7)
    tree = tree_of(T, n, 2) | torch.eye(T, dtype=torch.bool)
    length = torch.tensor([n, n // 2], dtype=torch.int32)
    want = ref.attend(x, k, v, length, tree=tree)["out"]
    spread = ref.attend(x, k, v.float().abs().to(cache), length, tree=tree)["out"]
    out = kv.attend(put(x), put(k), put(v), length.to(DEV), tree=put(tree))
    # a score's terms add up to less than 1/8: sums of D of them and a few roundings, and of 2^x; sums of n + T weights and
    # of their products
    assert float((x.float().abs().view(-1, D) @ k.float().abs().view(-1, D).t()).max()) / math.sqrt(D) < 0.125
    ds = (D + 16) * 2.0 ** -23 / 8 + 2.0 ** -21
    two = 2.0 ** -15 if cache == BF16 else 2.0 ** -21
    ref.within(out, want, want.abs() * ref.HALF[q] * (1 + 2.0 ** -10) + ref.TINY[q] + spread * (two + 2.0 ** -35 + 2 * ds + 2 * (n + T) * 2.0 ** -24), "out")
