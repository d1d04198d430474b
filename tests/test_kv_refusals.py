"""CPU tests of what the KV-cache operators' binding refuses, and says about it."""
import pytest
import torch

from lossless_bf16_tensor_amd import kv
from lossless_bf16_tensor_amd.uzip import UzipError

BF16 = torch.bfloat16


def operands():
    k, v = torch.zeros(2, 8, 2, 64, dtype=BF16), torch.zeros(2, 8, 2, 64, dtype=BF16)
    n = torch.zeros(2, dtype=torch.int32)
    q, new = torch.zeros(2, 1, 4, 64, dtype=BF16), torch.zeros(2, 1, 2, 64, dtype=BF16)
    return dict(k=k, v=v, n=n, q=q, new=new, new_v=new.clone(), score=torch.zeros(2, 2, 8), pos=torch.zeros(1, dtype=torch.int32), freq=kv.rope_freq(64),
                out=torch.zeros_like(q), lse=torch.zeros(2, 1, 4), k_out=torch.zeros(2, 4, 2, 64, dtype=BF16),
                v_out=torch.zeros(2, 4, 2, 64, dtype=BF16))


CALLS = dict(rope=lambda o: kv.rope(o["q"], o["pos"], o["freq"], out=o["out"]),
             append=lambda o: kv.append(o["q"], o["new"], o["new_v"], o["k"], o["v"], o["n"], o["freq"], out=o["out"]),
             attend=lambda o: kv.attend(o["q"], o["k"], o["v"], o["n"], score=o["score"], lse=o["lse"], out=o["out"]),
             evict=lambda o: kv.evict(o["k"], o["v"], o["score"], o["n"], 4, k_out=o["k_out"], v_out=o["v_out"]))


@pytest.mark.parametrize("call,names", [("rope", ("q", "freq", "out")), ("append", ("q", "new", "new_v", "k", "v", "freq", "out")),
                                        ("attend", ("q", "k", "v", "score", "lse", "out")), ("evict", ("k", "v", "score", "k_out", "v_out"))])
def test_tensors_that_require_a_gradient(call, names):
    """Refused, not silently detached; with gradients off, the call goes on to the next check."""
    for name in names:
        o = operands()
        o[name].requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            CALLS[call](o)
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            CALLS[call](o)
    with pytest.raises(ValueError, match="device tensors"):
        CALLS[call](operands())


def test_views_that_do_not_fit_are_named():
    """What the library refuses without a reason: off a 16-byte boundary, strides
    that are not multiples of 8, too far apart, empty, of a head dim that is none."""
    q = torch.zeros(2, 1, 4, 64, dtype=BF16)
    kv._fits(q, "q")
    for t, why in ((torch.zeros(q.numel() + 4, dtype=BF16)[4:].view(q.shape), "q does not start on a 16-byte"),
                   (torch.zeros(2, 1, 4, 68, dtype=BF16)[..., :64], "multiples of 8"),
                   (torch.empty(1, 2, 1, 1 << 26, dtype=BF16, device="meta")[..., :64], "below 2"),
                   (torch.zeros(2, 0, 4, 64, dtype=BF16), "q is empty"), (torch.zeros(2, 1, 4, 60, dtype=BF16), "multiple of 8"),
                   (torch.zeros(2, 1, 4, 264, dtype=BF16), "multiple of 8")):
        with pytest.raises(ValueError, match=why):
            kv._fits(t, "q")
        with pytest.raises(ValueError, match=why):
            kv._check(-1, "attend", x=q, q=t, out=None)
    with pytest.raises(UzipError, match="attend"):
        kv._check(-1, "attend", q=q)
    with pytest.raises(UzipError, match="attend"):
        kv._check(-2, "attend", q=torch.zeros(2, 1, 4, 60, dtype=BF16))


def test_strides_of_one_element_are_free():
    for t in (torch.zeros(1, 3, 1, 68, dtype=BF16)[:, :1, :, :64], torch.empty(1, 1, 1, 1 << 27, dtype=BF16, device="meta")[..., :64]):
        assert kv._strides(t) == (0, 0, 0)
        kv._fits(t, "q")


def test_no_heads():
    o = operands()
    with pytest.raises(ValueError, match="query heads"):
        kv.attend(o["q"], o["k"][:, :, :0], o["v"][:, :, :0], o["n"])


@pytest.mark.parametrize("page", [8, 24])
def test_pages_that_do_not_fit(page):
    o = operands()
    k, v = (torch.zeros(2, page, 2, 64, dtype=BF16) for _ in range(2))
    with pytest.raises(ValueError, match="power of two"):
        kv.attend(o["q"], k, v, o["n"], table=torch.zeros(2, 1, dtype=torch.int32))


def test_outputs_that_are_other_operands():
    """By their addresses, which the library sees: the caches' keys as values,
    turned queries over the new keys or values, kept keys as kept values."""
    import test_kv_host as host
    assert host.append(host.cache(v=1 << 20)) == host.EINVAL
    assert host.append(out=host.tensor(1 << 23), k=host.tensor(1 << 23)) == host.EINVAL
    assert host.append(out=host.tensor(1 << 23), v=host.tensor(1 << 23)) == host.EINVAL
    for k, v in ((1 << 26, 1 << 26), (1 << 21, 1 << 27), (1 << 26, 1 << 20)):
        assert host.evict(out=host.cache(k=k, v=v, tokens=16)) == host.EINVAL
