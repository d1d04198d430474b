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
