"""More of kv.verify, kv.fork and kv.copy_pages: what other tests do not reach."""
import pytest
import torch

from lossless_bf16_tensor_amd import kv
from test_gpu_kv_step import DEV, I32, check, check_fork

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


def test_pages_that_are_whole_for_some_and_partly_filled_for_others():
    """The same pages marked from all over the chip, as whole ones and as last
    ones: whole for any sequence, they are nobody's to fill on."""
    S, E, page, pages = 900, 40, 16, 3000
    g = torch.Generator().manual_seed(6)
    prefix = torch.randperm(pages, generator=g)[:E].to(I32)
    table = prefix.expand(S, E).contiguous()
    length = torch.randint(1, E * page, (S,), generator=g).to(I32)
    length[S // 2:] = (length[S // 2:] // page * page).clamp(min=page) - 3          # last pages partly filled, up to all of them
    table[::7, -1] = torch.randperm(pages, generator=g)[:len(table[::7])].to(I32)
    parent = torch.randint(0, S, (1500,), generator=g).to(I32)
    for held in (None, torch.rand(pages, generator=g) < 0.05):
        t, n, moves, left = check_fork(table, length, parent, pages, page, 20, held)
        assert int((moves[:, 0] >= 0).sum()) > 1000


def test_more_moves_than_a_launch_holds():
    """A table of moves that is padded, as compact's is, beyond 2^24 workgroups: its first, middle and last ones are made."""
    n = (1 << 24) + 3
    moves = torch.full((n, 2), -1, dtype=I32, device=DEV)
    real = {0: (1, 10), n // 2: (2, 11), (1 << 24) - 2: (3, 12), (1 << 24) - 1: (4, 13), 1 << 24: (5, 14), n - 1: (6, 15)}
    pool = torch.arange(20 * 16 * 3, device=DEV).view(20, 16, 3).to(torch.int8)
    want = pool.clone()
    for i, (a, b) in real.items():
        moves[i] = torch.tensor([a, b], dtype=I32)
        want[b] = pool[a]
    kv.copy_pages(moves, pool)
    assert torch.equal(pool, want)
