"""More of kv.verify, kv.fork and kv.copy_pages: what other tests do not reach."""
import pytest
import torch

from test_gpu_kv_step import I32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_token_again_right_behind_its_rejection(dtype):
    """Pairs of children with one token: the first is rejected, and the second,
    which any probability would accept, is the next to be looked at."""
    B, pairs, V = 5, 150, 400
    g = torch.Generator().manual_seed(3)
    p = torch.softmax(torch.randn(B, 1 + 2 * pairs, V, generator=g), -1).to(dtype)
    tokens = torch.zeros(B, 1 + 2 * pairs, dtype=I32)
    u = torch.zeros(B, 1 + 2 * pairs)
    u[:, 0], u[:, 1::2] = torch.rand(B, generator=g), 1 - 2.0 ** -24
    for b in range(B):
        tokens[b, 1:] = torch.randperm(V, generator=g)[:pairs].repeat_interleave(2).int()
    found = check(dict(tokens=tokens, target=p, uniform=u, draft=None, parent=torch.tensor([-1] + [0] * (2 * pairs), dtype=I32)))
    assert {n for _, n, _ in found} == {1}
