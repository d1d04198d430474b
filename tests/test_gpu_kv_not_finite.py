"""kv.attend over values that are not finite and whose keys carry no weight."""
import math

import pytest
import torch

from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV, E5M2, F16, bits

pytestmark = pytest.mark.gpu


def bad_value(v, at, value):
    bits(v)[at] = bits(torch.full((1,), value).to(v.dtype)).to(v.device)


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2)])
@pytest.mark.parametrize("T,hq", [(2, 1), (3, 8), (40, 1)])
@pytest.mark.parametrize("n", [0, 20, 3000, 40000])
def test_rows_of_minus_infinity_are_zeros(dtype, cache, T, hq, n):
    """Every seen score is -inf and a drafted value infinite or NaN: zeros and
    -inf, in one part (a short cache) and in many."""
    g = torch.Generator().manual_seed(n + T)
    q = torch.randn(1, T, hq, 64, generator=g)
    q[..., 0] = 1.0
    k, v = (torch.randn(1, n + T, 1, 64, generator=g) for _ in range(2))
    k[..., 0] = -math.inf
    k, v = k.to(cache), v.to(cache)
    bad_value(v, (0, n, 0, 5), math.inf)
    bad_value(v, (0, n, 0, 6), math.nan)
    bad_value(v, (0, n + 1, 0, 7), -math.inf)
    lse = torch.full((1, T, hq), 2.0, device=DEV)
    score = torch.zeros(1, 1, n + T, device=DEV)
    out = kv.attend(q.to(dtype).to(DEV), k.to(DEV), v.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), lse=lse, score=score)
    assert not out.any() and (lse == -math.inf).all() and not score.any()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2)])
@pytest.mark.parametrize("n", [20, 3000, 40000])
@pytest.mark.parametrize("where", ["drafted", "cached"])
def test_an_infinite_value_of_a_weight_near_zero_shows(dtype, cache, n, where):
    """A seen value that is not finite leaves its element of the output not
    finite, in one part and in many, though its key's weight rounds to zero;
    the others are as they would be."""
    g = torch.Generator().manual_seed(n)
    q = torch.randn(1, 2, 4, 64, generator=g)
    q[..., 0] = 1.0
    k, v = (torch.randn(1, n + 2, 1, 64, generator=g) for _ in range(2))
    key = n if where == "drafted" else n // 2
    k[..., 0] = 0.0
    k[:, key, :, 0] = -8192.0
    q, k, v = q.to(dtype).to(DEV), k.to(cache).to(DEV), v.to(cache).to(DEV)
    length = torch.tensor([n], dtype=torch.int32, device=DEV)
    want = kv.attend(q, k, v, length)
    assert torch.isfinite(want).all()
    bad_value(v, (0, key, 0, 9), math.inf)
    got = kv.attend(q, k, v, length)
    rest = [d for d in range(64) if d != 9]
    assert not torch.isfinite(got[..., 9]).any()
    assert torch.equal(got[..., rest], want[..., rest])


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2), (F16, E5M2)])
@pytest.mark.parametrize("B,T,hq,H,D,n", [(1, 1, 1, 1, 64, 5), (2, 1, 8, 2, 128, 3000), (1, 6, 4, 1, 128, 900), (1, 3, 16, 2, 256, 500),
                                          (16, 66, 32, 32, 64, 2334)])
@pytest.mark.parametrize("equal", [False, True])
def test_infinite_values_of_cached_tokens(dtype, cache, B, T, hq, H, D, n, equal):
    """Infinities that every query sees, of weights that are powers of two
    (equal keys) and any others: infinities of their sign, NaN where both signs
    meet, and the other elements as they would be."""
    g = torch.Generator().manual_seed(n + D)
    q = torch.randn(B, T, hq, D, generator=g).to(dtype).to(DEV)
    k = torch.randn(B, n + T, H, D, generator=g) * (0.0 if equal else 0.5)
    v = torch.randn(B, n + T, H, D, generator=g).to(cache)
    k, v = k.to(cache).to(DEV), v.to(DEV)
    length = torch.full((B,), n, dtype=torch.int32, device=DEV)
    want = kv.attend(q, k, v, length)
    assert torch.isfinite(want).all()
    for key, d, value in ((0, 3, math.inf), (n // 2, 4, -math.inf), (n - 1, 60, math.inf), (n - 1, 5, math.inf), (1, 5, -math.inf), (2, 6, math.nan)):
        bits(v)[:, key, :, d] = bits(torch.full((1,), value).to(cache)).to(DEV)
    got = kv.attend(q, k, v, length)
    assert (got[..., 3] == math.inf).all() and (got[..., 4] == -math.inf).all() and (got[..., 60] == math.inf).all()
    assert torch.isnan(got[..., 5:7]).all()
    rest = [d for d in range(D) if d not in (3, 4, 5, 6, 60)]
    assert torch.equal(got[..., rest], want[..., rest])
