"""kv.rope and kv.append leave what they do not turn as it is, bit for bit, NaN
of every payload included."""
import pytest
import torch

from lossless_bf16_tensor_amd import kv
from test_gpu_kv_attend import BF16, DEV, F16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rot", [2, 20, 24, 60, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_value_behind_the_turned_ones(dtype, rot, interleaved):
    words = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = words.view(256, 256)[:, :, None].expand(256, 256, 8).reshape(4, 128, 8, 128).contiguous()
    x = torch.cat((x, x.roll(37, 1)), -1).view(dtype).to(DEV)                    # [4, 128, 8, 256]
    pos = torch.arange(128, dtype=torch.int32, device=DEV)
    freq = kv.rope_freq(rot).to(DEV)
    got = kv.rope(x, pos, freq, interleaved=interleaved)
    assert torch.equal(got.view(torch.int16)[..., rot:], x.view(torch.int16)[..., rot:])
    kc, vc = (torch.zeros(4, 130, 8, 256, dtype=dtype, device=DEV) for _ in range(2))
    n = torch.full((4,), 2, dtype=torch.int32, device=DEV)
    q = kv.append(x, x, x, kc, vc, n, freq, pos=pos, interleaved=interleaved)
    assert torch.equal(q.view(torch.int16), got.view(torch.int16)) and torch.equal(kc[:, 2:].view(torch.int16), got.view(torch.int16))
    assert torch.equal(vc[:, 2:].view(torch.int16), x.view(torch.int16))
