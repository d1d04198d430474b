"""More CPU tests of the host side of the operators over 8-bit caches and pages.
Every call below returns before it touches the GPU."""
from lossless_bf16_tensor_amd import kv
from test_kv_host import EINVAL, ENOSPC, cache, rope_args
from test_kv_step_host import append, attend, scales


def test_scales_lead_to_no_element_2_to_the_30():
    c = cache(dtype=4, heads=4, table=1 << 23, page=32, pages=3, tokens=64)
    last = lambda s: 2 * s[0] + s[1] + 3 * s[2]  # noqa: E731
    near, far = ((2 ** 30 - 8) // 2, 4, 1), ((2 ** 30 - 8) // 2, 5, 1)
    assert last(near) == 2 ** 30 - 1 and last(far) == 2 ** 30
    for name in ("ks", "vs"):
        assert attend(c, scales(**{name: near}), ws_bytes=0) == ENOSPC
        assert attend(c, scales(**{name: far}), ws_bytes=0) == EINVAL
        assert append(c, scales(**{name: far})) == EINVAL


def test_more_workgroups_than_a_launch_holds():
    """Refused before anything runs, not when a later kernel cannot be launched."""
    many = dict(seqs=65535, heads=512, dim=8, ks=(4096, 4096, 8), vs=(4096, 4096, 8), tokens=1)
    c = cache(dtype=4, **many)
    assert attend(c, scales(ks=(512, 512, 1), vs=(512, 512, 1)), T=1, heads=512) == EINVAL
    args = kv._ATTEND.pack(1 << 22, 4096, 4096, 8, 1 << 21, 4096, 4096, 8, 0, 0, 0, 0, 1 << 24, 0, 0, 0, 0, 0, 1, 512, 0.1, 0, 0)
    assert kv.lib().uzip_kv_attend(cache(**many), args, 1 << 25, 1 << 40, None) == EINVAL
    # ... for the accumulated weights
    long = dict(seqs=4096, heads=2, dim=8, ks=(16, 16, 8), vs=(16, 16, 8), tokens=1 << 24)
    args = kv._ATTEND.pack(1 << 22, 16, 16, 8, 1 << 21, 16, 16, 8, 0, 1 << 23, 0, 0, 1 << 24, 0, 0, 0, 0, 0, 1, 2, 0.1, 1 << 24, 0)
    assert kv.lib().uzip_kv_attend(cache(**long), args, 1 << 25, 1 << 50, None) == EINVAL
    one = dict(seqs=1, heads=1, dim=8, ks=(0, 8, 8), vs=(0, 8, 8), tokens=1 << 30)
    assert append(cache(dtype=4, **one), scales(ks=(0, 1, 1), vs=(0, 1, 1)), T=(1 << 28) + 16, heads=1) == EINVAL
    wide = dict(seqs=65535, heads=4096, dim=256, ks=(1 << 20, 1 << 20, 256), vs=(1 << 20, 1 << 20, 256), tokens=1)
    assert kv.lib().uzip_kv_accept(cache(**wide), kv._ACCEPT.pack(1 << 24, 1 << 24, 4, 1 << 24, 4, 0), None) == EINVAL


def test_more_workgroups_than_a_launch_holds_without_scales():
    rope = lambda T, H: kv.lib().uzip_kv_rope(kv._TENSOR.pack(1 << 22, 0, H * 256, 256), kv._TENSOR.pack(1 << 23, 0, H * 256, 256), 0, 1, T, H, 256,  # noqa: E731
                                              rope_args(rot=256), None)
    assert rope(1 << 25, 64) == EINVAL
    c = cache(seqs=1, heads=16, dim=256, ks=(0, 4096, 256), vs=(0, 4096, 256), tokens=1 << 30)
    args = kv._APPEND.pack(*(0,) * 8, 1 << 22, 0, 4096, 256, 1 << 23, 0, 4096, 256, 1 << 24, 0, 0, 1 << 26, 0, 0)
    assert kv.lib().uzip_kv_append(c, args, None, None) == EINVAL

    def evict(seqs, heads, tokens, keep, ws=1 << 25):
        k = dict(seqs=seqs, heads=heads, dim=8, ks=(heads * 8, heads * 8, 8), vs=(heads * 8, heads * 8, 8))
        args = kv._EVICT.pack(1 << 26, 0, 0, 1 << 24, 1 << 23, 1 << 23, 1 << 23, keep, 0, 0, tokens)
        return kv.lib().uzip_kv_evict(cache(**k, tokens=tokens), cache(**dict(k, k=1 << 27, v=1 << 28), tokens=keep), args, ws, 1 << 60, None)
    assert evict(65535, 65, 16, 1) == EINVAL                          # a workgroup of 1024 a row
    assert evict(1024, 64, 1 << 20, 1) == EINVAL                      # ... for each 8192 tokens of one
    assert evict(1024, 64, 1 << 20, 1 << 19) == EINVAL
