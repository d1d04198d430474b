"""Calls that the KV-cache operators refuse on the device, before anything is
launched, and the reason they give."""
import pytest
import torch

from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV

pytestmark = pytest.mark.gpu


def operands():
    mk = lambda *s: torch.zeros(*s, dtype=BF16, device=DEV)  # noqa: E731
    return dict(q=mk(2, 1, 4, 64), new=mk(2, 1, 2, 64), new_v=mk(2, 1, 2, 64), k=mk(2, 8, 2, 64), v=mk(2, 8, 2, 64), out=mk(2, 1, 4, 64),
                k_out=mk(2, 4, 2, 64), v_out=mk(2, 4, 2, 64), n=torch.zeros(2, dtype=torch.int32, device=DEV),
                score=torch.zeros(2, 2, 8, device=DEV), pos=torch.zeros(1, dtype=torch.int32, device=DEV), freq=kv.rope_freq(64, device=DEV))


CALLS = dict(rope=(lambda o: kv.rope(o["q"], o["pos"], o["freq"], out=o["out"]), "q out"),
             append=(lambda o: kv.append(o["q"], o["new"], o["new_v"], o["k"], o["v"], o["n"], o["freq"], out=o["out"]), "q new new_v k v out"),
             attend=(lambda o: kv.attend(o["q"], o["k"], o["v"], o["n"], out=o["out"]), "q k v out"),
             evict=(lambda o: kv.evict(o["k"], o["v"], o["score"], o["n"], 4, k_out=o["k_out"], v_out=o["v_out"]), "k v k_out v_out"))


@pytest.mark.parametrize("call", CALLS)
def test_views_that_do_not_fit(call):
    f, names = CALLS[call]
    f(operands())
    for name in names.split():
        o = operands()
        t = o[name]
        o[name] = torch.zeros(t.numel() + 4, dtype=BF16, device=DEV)[4:].view(t.shape)
        with pytest.raises(ValueError, match="16-byte"):
            f(o)
        o[name] = torch.zeros(*t.shape[:3], 68, dtype=BF16, device=DEV)[..., :64]
        with pytest.raises(ValueError, match="multiples of 8"):
            f(o)


@pytest.mark.parametrize("call", CALLS)
def test_nothing_at_all(call):
    """No sequences, and no tokens."""
    f, names = CALLS[call]
    for cut in (lambda t: t[:0], lambda t: t[:, :0] if t.dim() == 4 else t):
        o = {name: cut(t) if t.dim() > 1 or name == "n" else t for name, t in operands().items()}
        with pytest.raises(ValueError):
            f(o)
