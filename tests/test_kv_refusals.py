"""CPU tests of what the KV-cache operators' binding refuses, and says about it."""
import pytest
import torch

from lossless_bf16_tensor_amd import kv

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


def moved(t, by):
    """t's values `by` elements behind the start of its memory."""
    whole = torch.zeros(t.numel() + by, dtype=t.dtype)
    return whole[by:].view(t.shape)


@pytest.mark.parametrize("call,names", [("rope", ("q", "out")), ("append", ("q", "new", "new_v", "k", "v", "out")), ("attend", ("q", "k", "v", "out")),
                                        ("evict", ("k", "v"))])
def test_views_that_do_not_fit_are_named(call, names):
    """Off a 16-byte boundary, of strides that are not multiples of 8, empty, of
    a head dim that is none: each says so. (Outputs are looked at last, on the
    device: their rules are the inputs'.)"""
    for name in names:
        if name == "out":
            continue
        o = operands()
        o[name] = moved(o[name], 4)
        with pytest.raises(ValueError, match="16-byte"):
            CALLS[call](o)
        o = operands()
        shape = o[name].shape
        o[name] = torch.zeros(shape[0], shape[1], shape[2], 68, dtype=BF16)[..., :64]
        with pytest.raises(ValueError, match="multiples of 8"):
            CALLS[call](o)


@pytest.mark.parametrize("shape,why", [((2, 0, 4, 64), "empty"), ((2, 1, 4, 60), "multiple of 8"), ((2, 1, 4, 264), "multiple of 8"), ((2, 4, 64), "four dims")])
def test_shapes_that_do_not_fit_are_named(shape, why):
    q = torch.zeros(shape, dtype=BF16)
    with pytest.raises(ValueError, match=why):
        kv._strides(q, "q")
    if len(shape) == 4:
        with pytest.raises(ValueError, match=why):
            kv.rope(q, torch.zeros(shape[1], dtype=torch.int32), kv.rope_freq(8))
        with pytest.raises(ValueError, match=why):
            kv.attend(q, torch.zeros(2, 8, 2, shape[3], dtype=BF16), torch.zeros(2, 8, 2, shape[3], dtype=BF16), torch.zeros(2, dtype=torch.int32))


def test_strides_of_one_element_are_free():
    whole = torch.zeros(1, 3, 1, 68, dtype=BF16)
    assert kv._strides(whole[:, :1, :, :64], "q") == (0, 0, 0)
    assert kv._strides(torch.empty(1, 1, 1, 1 << 27, dtype=BF16, device="meta")[..., :64], "q") == (0, 0, 0)
    with pytest.raises(ValueError, match="below 2"):
        kv._strides(torch.empty(1, 2, 1, 1 << 26, dtype=BF16, device="meta")[..., :64], "q")


def test_pages_that_do_not_fit_are_named():
    o = operands()
    with pytest.raises(ValueError, match="power of two"):
        kv.attend(o["q"], o["k"], o["v"], o["n"], table=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="power of two"):
        kv.attend(o["q"], torch.zeros(2, 24, 2, 64, dtype=BF16), torch.zeros(2, 24, 2, 64, dtype=BF16), o["n"], table=torch.zeros(2, 1, dtype=torch.int32))


def test_outputs_that_are_other_operands():
    """By their addresses, which the library sees: the caches' keys as values,
    turned queries over the new keys or values, kept keys as kept values."""
    import test_kv_host as host
    assert host.append(host.cache(v=1 << 20)) == host.EINVAL
    assert host.append(out=host.tensor(1 << 23), k=host.tensor(1 << 23)) == host.EINVAL
    assert host.append(out=host.tensor(1 << 23), v=host.tensor(1 << 23)) == host.EINVAL
    for k, v in ((1 << 26, 1 << 26), (1 << 21, 1 << 27), (1 << 26, 1 << 20)):
        assert host.evict(out=host.cache(k=k, v=v, tokens=16)) == host.EINVAL
