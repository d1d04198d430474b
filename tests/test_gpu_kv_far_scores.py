"""kv.attend with scores so large that a step of binary32 there is more than a
factor of two in the weights."""
import pytest
import torch

import kv_reference as ref
from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV, E5M2, F16, put

pytestmark = pytest.mark.gpu

Q = 165 / 128                                     # its products with the scale are rounded in binary32


@pytest.mark.parametrize("dtype,cache,size,key", [(BF16, BF16, 40, 0), (BF16, BF16, 20, 0), (F16, F16, 15, 14), (F16, F16, 12, 8), (BF16, E5M2, 60, 2),
                                                  (F16, E5M2, 15, 13), (BF16, BF16, 100, 20)])
@pytest.mark.parametrize("T,hq,n,D", [(1, 1, 40, 64), (3, 8, 700, 128), (20, 2, 5000, 64), (70, 1, 3000, 128), (9, 1, 100, 256)])
def test_the_largest_score_takes_all(dtype, cache, size, key, T, hq, n, D):
    """Scores are whole multiples, -4 to 3, of one number, the largest of
    one cached key alone; so its weight is 1, all others are 0, and the output
    is its values. Once all are negative, once the largest comes last. lse is
    the largest score: two products rounded to binary32."""
    g = torch.Generator().manual_seed(n)
    k = torch.randn(1, n + T, 1, D, generator=g) * 0.0
    k[..., 0] = torch.randint(-3, 1, (1, n + T, 1), generator=g) * 2.0 ** key
    v = torch.randn(1, n + T, 1, D, generator=g).to(cache)
    q = torch.zeros(1, T, hq, D)
    q[..., 0] = Q * 2.0 ** size
    for most, shift in ((3, 0), (-1, -1)):
        for at in (0, n // 2, n - 1):
            x = k.clone()
            x[..., 0] += shift * 2.0 ** key
            x[0, at, 0, 0] = most * 2.0 ** key
            if shift:                             # -4 to -2, but for one of -1
                x[..., 0] = torch.where(x[..., 0] == -1.0 * 2.0 ** key, -2.0 * 2.0 ** key, x[..., 0])
                x[0, at, 0, 0] = -1.0 * 2.0 ** key
            lse = torch.empty(1, T, hq, device=DEV)
            out = kv.attend(put(q.to(dtype)), put(x.to(cache)), put(v), torch.tensor([n], dtype=torch.int32, device=DEV), scale=0.3, lse=lse)
            assert torch.equal(out.cpu().double(), v[0, at].double().expand(1, T, hq, D))
            want = torch.full((1, T, hq), torch.tensor(0.3).double() * most * Q * 2.0 ** (size + key), dtype=torch.float64)
            ref.within(lse, want, want.abs() * 2.0 ** -21, "lse")


@pytest.mark.parametrize("B,H", [(16, 32)])
def test_the_largest_score_takes_all_of_shared_keys(B, H):
    T, S, D = 66, 2400, 64
    g = torch.Generator().manual_seed(5)
    k = torch.zeros(B, S, H, D)
    k[..., 0] = torch.randint(-3, 1, (B, S, H), generator=g) * 2.0 ** 14
    at = torch.randint(0, S - T, (B, H), generator=g)
    k[torch.arange(B)[:, None], at, torch.arange(H), 0] = 2.0 ** 14
    v = torch.randn(B, S, H, D, generator=g).to(F16)
    q = torch.zeros(B, T, H, D, dtype=F16)
    q[..., 0] = Q * 2.0 ** 15
    out = kv.attend(put(q), put(k.to(F16)), put(v), torch.full((B,), S - T, dtype=torch.int32, device=DEV), scale=0.3)
    want = v[torch.arange(B)[:, None], at, torch.arange(H)]
    assert torch.equal(out.cpu(), want[:, None].expand(B, T, H, D))
