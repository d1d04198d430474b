"""kv.rope and kv.append against their 64-bit forms."""
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


def positions(B, T, seed, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (B, T), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 2), (8, 8), (64, 64), (64, 32), (80, 80), (96, 20), (128, 128), (128, 48), (256, 256),
                                   (256, 6), (128, 8), (248, 248)])
def test_rope(dtype, interleaved, D, rot):
    g = torch.Generator().manual_seed(D + rot)
    for B, T, H in ((1, 1, 1), (2, 3, 5), (3, 37, 9)):
        x = torch.randn(B, T, H, D, generator=g).to(dtype)
        pos = positions(B, T, T)
        freq = kv.rope_freq(rot)
        for inverse in (False, True):
            want = ref.turned(x, pos, freq, 1.25, interleaved, inverse)
            got = kv.rope(x.to(DEV), pos.to(DEV), freq.to(DEV), amplitude=1.25, interleaved=interleaved, inverse=inverse)
            ref.within(got, want, ref.rope_bound(x, want, freq, 1.25, dtype), f"{B} {T} {H} inverse {inverse}")
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (20, False), (20, True), (64, False)])
def test_rope_in_place_and_in_views(rot, interleaved):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn(2, 6, 50, 144, generator=g).to(BF16)
    pos = positions(1, 50, 3)[0]
    freq = kv.rope_freq(rot).to(DEV)
    want = ref.turned(x[..., 8:136].transpose(1, 2), pos.expand(2, 50), freq.cpu(), 1.0, interleaved)
    whole = x.to(DEV)
    view = whole[..., 8:136].transpose(1, 2)      # [sequences, tokens, heads, dim] of a heads-first tensor
    got = kv.rope(view, pos.to(DEV), freq, interleaved=interleaved, out=view)
    assert got.data_ptr() == view.data_ptr()
    ref.within(view, want, ref.rope_bound(x[..., 8:136].transpose(1, 2), want, freq, 1.0, BF16))
    assert torch.equal(whole[..., :8].cpu(), x[..., :8]) and torch.equal(whole[..., 136:].cpu(), x[..., 136:])


@pytest.mark.parametrize("H,D,rot,interleaved", [(1, 8, 8, False), (1, 64, 64, True), (2, 128, 96, False), (1, 256, 256, False), (3, 72, 20, True),
                                                (5, 64, 20, False)])
def test_many_tokens_of_few_heads(H, D, rot, interleaved):
    """Several tokens a workgroup, the last one not full; and the same of an append."""
    g = torch.Generator().manual_seed(H + rot)
    B, T = 3, 3457
    x = torch.randn(B, T, H, D, generator=g).to(BF16)
    pos = positions(B, T, 4)
    freq = kv.rope_freq(rot)
    want = ref.turned(x, pos, freq, 1.0, interleaved)
    got = kv.rope(x.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved)
    ref.within(got, want, ref.rope_bound(x, want, freq, 1.0, BF16))
    kc, vc = (torch.zeros(B, T + 5, H, D, dtype=BF16, device=DEV) for _ in range(2))
    n = torch.tensor([0, 5, 2], dtype=torch.int32)
    drafted = torch.tensor([T, T, 1000], dtype=torch.int32)
    q = kv.append(x.to(DEV), x.to(DEV), x.to(DEV), kc, vc, n.to(DEV), freq.to(DEV), pos=pos.to(DEV), drafted=drafted.to(DEV), interleaved=interleaved)
    assert torch.equal(q, got)
    for b in range(B):
        m, k = int(drafted[b]), int(n[b])
        assert torch.equal(kc[b, k:k + m], got[b, :m]) and torch.equal(vc[b, k:k + m].cpu(), x[b, :m])
        assert not kc[b, :k].any() and not kc[b, k + m:].any() and not vc[b, k + m:].any()


def test_gradient_of_rope_by_differences():
    """The inverse with the same amplitude is the transposed map: <w, R x> = <R^-1 w, x>, and R x changes along d by R d."""
    g = torch.Generator().manual_seed(0)
    x, w = (torch.randn(1, 5, 2, 64, generator=g).to(F16) for _ in range(2))
    pos, freq = positions(1, 5, 1), kv.rope_freq(48)
    args = dict(amplitude=0.75)
    y = kv.rope(x.to(DEV), pos.to(DEV), freq.to(DEV), **args).cpu().double()
    grad = kv.rope(w.to(DEV), pos.to(DEV), freq.to(DEV), inverse=True, **args).cpu().double()
    # each of the 640 terms is off by at most half a step of FP16 on either side
    size = float((w.double().abs() * y.abs()).sum() + (grad.abs() * x.double().abs()).sum())
    assert abs(float((w.double() * y).sum() - (grad * x.double()).sum())) <= 2.0 ** -11 * 1.01 * size
    for at in ((0, 0, 0, 0), (0, 3, 1, 30), (0, 4, 0, 60)):
        x2 = x.clone()
        step = 0.25
        x2[at] += step
        step = float(x2[at] - x[at])
        y2 = kv.rope(x2.to(DEV), pos.to(DEV), freq.to(DEV), **args).cpu().double()
        slope = float((w.double() * (y2 - y)).sum()) / step
        # only the pair of `at` moves: two outputs, rounded to half a step before and after, and the gradient itself
        moved = (y2 != y)
        room = float((w.double().abs() * moved * (y.abs() + y2.abs())).sum()) * 2.0 ** -11 / step + abs(float(grad[at])) * 2.0 ** -11
        assert abs(slope - float(grad[at])) <= 1.01 * room + 2.0 ** -20


@pytest.mark.parametrize("scaling", [dict(), dict(linear=4.0), dict(ntk=8.0), dict(bands=(8.0, 8192, 1.0, 32.0))])
def test_far_positions(scaling):
    """The angle's fraction of a turn is taken in 64 bits: no loss at positions up to 2^31."""
    x = torch.randn(1, 4, 1, 128, generator=torch.Generator().manual_seed(2)).to(F16)
    pos = torch.tensor([[0, 1 << 24, (1 << 31) - 1, -(1 << 20)]], dtype=torch.int32)
    freq = kv.rope_freq(128, 500000.0, **scaling)
    want = ref.turned(x, pos, freq)
    ref.within(kv.rope(x.to(DEV), pos.to(DEV), freq.to(DEV)), want, ref.rope_bound(x, want, freq, 1.0, F16))


CASES = [  # B, T, Hq, H, D, S, layout, rot, interleaved
    (1, 1, 4, 1, 128, 9, "shd", 128, False), (3, 5, 8, 2, 64, 40, "hsd", 64, True), (2, 33, 6, 3, 80, 70, "paged16", 20, False),
    (4, 3, 7, 7, 128, 33, "paged32", 48, True), (2, 300, 4, 2, 256, 310, "shd", 256, False), (1, 2, 2, 2, 8, 7, "shd", 0, False)]


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E5M2), (F16, E5M2)])
@pytest.mark.parametrize("case", CASES)
def test_append(dtype, cache, case):
    B, T, hq, H, D, S, layout, rot, interleaved = case
    g = torch.Generator().manual_seed(T + D)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = mk(B, T, hq, D).to(dtype), mk(B, T, H, D).to(dtype), mk(B, T, H, D).to(dtype)
    table = None
    if layout.startswith("paged"):
        page = int(layout[5:])
        per = -(-S // page)
        table = torch.randperm(B * per + 1, generator=g)[:B * per].view(B, per).to(torch.int32)
        table[0, 0] = -1                          # the first page of sequence 0 is absent
        kc, vc = mk(B * per + 1, page, H, D).to(cache), mk(B * per + 1, page, H, D).to(cache)
    else:
        kc, vc = mk(B, S, H, D).to(cache), mk(B, S, H, D).to(cache)
    cap = S if table is None else table.shape[1] * kc.shape[1]
    length = torch.randint(-1, cap + 1, (B,), generator=g, dtype=torch.int32)      # past the ends too
    drafted = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    drafted[-1] = T
    freq = kv.rope_freq(rot) if rot else None
    pos = length[:, None] + torch.arange(T, dtype=torch.int32)
    turn = (lambda x: ref.turned(x, pos, freq, 1.1, interleaved)) if rot else (lambda x: x.to(ref.F64))
    want_q, want_k, want_v = turn(q), kc.to(ref.F64), vc.to(ref.F64)
    k_bound, v_bound = torch.zeros_like(want_k), torch.zeros_like(want_v)
    left = torch.ones(want_k.shape[:2], dtype=torch.bool)
    new_k = turn(k)
    kb = ref.rope_bound(k, new_k, freq, 1.1, cache) if rot or cache == E5M2 else torch.zeros_like(new_k)
    vb = v.to(ref.F64).abs() * ref.HALF[cache] + ref.TINY[cache] if cache == E5M2 else torch.zeros_like(v, dtype=ref.F64)
    for b in range(B):
        for t in range(int(drafted[b])):
            slot = int(length[b]) + t
            if not 0 <= slot < cap:
                continue
            at = (b, slot)
            if table is not None:
                at = (int(table[b, slot // kc.shape[1]]), slot % kc.shape[1])
                if at[0] < 0:
                    continue
            left[at] = False
            want_k[at], want_v[at], k_bound[at], v_bound[at] = new_k[b, t], v[b, t].to(ref.F64), kb[b, t], vb[b, t]
    if layout == "hsd":
        dk, dv = (bits(t).transpose(1, 2).contiguous().to(DEV).transpose(1, 2).view(cache) for t in (kc, vc))
    else:
        dk, dv = kc.to(DEV), vc.to(DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    given = dev(pos) if T % 2 else None           # the default is the same
    got = kv.append(dev(q), dev(k), dev(v), dk, dv, dev(length), dev(freq), pos=given, table=dev(table), drafted=dev(drafted),
                    amplitude=1.1, interleaved=interleaved)
    ref.within(got, want_q, ref.rope_bound(q, want_q, freq, 1.1, dtype) if rot else torch.zeros(()), "q")
    ref.within(dk.float(), want_k, k_bound, "k")
    ref.within(dv.float(), want_v, v_bound, "v")
    for got, was in ((dk, kc), (dv, vc)):         # the other rows as they were
        assert torch.equal(got.cpu().view(torch.uint8)[left], was.view(torch.uint8)[left])
    # without queries
    dk2, dv2 = dev(kc), dev(vc)
    assert kv.append(None, dev(k), dev(v), dk2, dv2, dev(length), dev(freq), table=dev(table), drafted=dev(drafted),
                     amplitude=1.1, interleaved=interleaved) is None
    assert torch.equal(bits(dk2), bits(dk)) and torch.equal(bits(dv2), bits(dv))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_value_rounds_to_e5m2_as_torch_rounds_it(dtype):
    words = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = words.view(dtype).view(1, 256, 1, 256).to(DEV)
    kc = torch.zeros(1, 256, 1, 256, dtype=E5M2, device=DEV)
    vc = torch.zeros_like(kc)
    kv.append(None, x, x, kc, vc, torch.zeros(1, dtype=torch.int32, device=DEV))
    want = x.float().to(E5M2).float()
    for got in (kc.float(), vc.float()):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


def test_append_in_a_graph():
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(3, 1, h, 128, generator=g).to(BF16).to(DEV) for h in (8, 2, 2))
    kc, vc = (torch.zeros(3, 64, 2, 128, dtype=BF16, device=DEV) for _ in range(2))
    n = torch.zeros(3, dtype=torch.int32, device=DEV)
    freq = kv.rope_freq(128).to(DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.append(q, k, v, kc, vc, n, freq, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.append(q, k, v, kc, vc, n, freq, out=out)
    for step in range(4):
        n.copy_(torch.tensor([step, 60 + step, 2 * step], dtype=torch.int32))
        q.copy_(torch.randn(3, 1, 8, 128, generator=g).to(BF16))
        k2, v2 = kc.clone(), vc.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kv.append(q, k, v, k2, v2, n, freq)) and torch.equal(kc, k2) and torch.equal(vc, v2)
    assert math.isfinite(float(kc.float().sum()))
