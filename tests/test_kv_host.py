"""CPU tests of the KV-cache operators' host side: symbols, structures, sizes,
refusals (every call below returns before it touches the GPU), and the rotary
frequencies."""
import ctypes
import math
import os
import re
import struct

import pytest
import torch

from lossless_bf16_tensor_amd import kv, uzip

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, ENOSPC = -1, -2


def test_every_declared_symbol_is_exported():
    src = open(os.path.join(ROOT, "include", "uzip_kv.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = set(re.findall(r"\b(uzip_kv_[a-z0-9_]+)\s*\(", src))
    assert declared == set(kv.EXPORTS)
    assert all(hasattr(kv.lib(), name) for name in declared)


CACHE = dict(k=1 << 20, v=1 << 21, table=0, ks=(0, 512, 128), vs=(0, 512, 128), ts=0, dtype=0, seqs=1, heads=4, dim=128,
             tokens=64, page=0, pages=0, reserved=0)


def cache(**kw):
    c = dict(CACHE, **kw)
    return kv._CACHE.pack(c["k"], c["v"], c["table"], *c["ks"], *c["vs"], c["ts"], c["dtype"], c["seqs"], c["heads"], c["dim"],
                          c["tokens"], c["page"], c["pages"], c["reserved"])


def tensor(data=1 << 22, stride=(0, 1024, 128)):
    return kv._TENSOR.pack(data, *stride)


BAD_CACHES = [dict(k=0), dict(v=0), dict(k=(1 << 20) + 8), dict(ks=(0, 512, 100)), dict(vs=(0, -512, 128)), dict(ks=(0, 1 << 26, 128)),
              dict(dtype=3), dict(seqs=0), dict(seqs=65536), dict(heads=0), dict(dim=0), dict(dim=100), dict(dim=264),
              dict(tokens=0), dict(tokens=(1 << 30) + 1), dict(reserved=1),
              dict(table=1 << 23, page=16, pages=0), dict(table=1 << 23, page=8, pages=4), dict(table=1 << 23, page=24, pages=4),
              dict(table=1 << 23, page=128, pages=4), dict(table=(1 << 23) + 2, page=16, pages=4),
              dict(table=1 << 23, page=16, pages=4, ts=-1)]


def attend(c=None, q=None, out=None, lse=0, score=0, ss=(256, 64), length=1 << 24, drafted=0, tree=0, ts=(0, 4), dtype=0, T=4,
           heads=8, scale=0.1, seen=64, reserved=0, ws=1 << 25, ws_bytes=1 << 40):
    args = kv._ATTEND.pack(*struct.unpack("=Q3q", q or tensor()), *struct.unpack("=Q3q", out or tensor(1 << 21)), lse, score, *ss, length,
                           drafted, tree, *ts, dtype, T, heads, scale, seen, reserved)
    return kv.lib().uzip_kv_attend(c or cache(), args, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(bad):
    c = cache(**bad)
    assert attend(c) == EINVAL
    assert append(c) == EINVAL
    assert evict(c) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=tensor(0)), dict(q=tensor(8)), dict(q=tensor(stride=(0, 4, 8))), dict(out=tensor(0)), dict(out=tensor(stride=(0, -8, 8))),
    dict(length=0), dict(length=2), dict(drafted=2), dict(lse=1), dict(score=3), dict(score=1 << 20, ss=(-1, 64)),
    dict(tree=1 << 20, ts=(-4, 4)), dict(dtype=1), dict(dtype=2), dict(T=0), dict(T=(1 << 20) + 1), dict(heads=0), dict(heads=6),
    dict(heads=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=2.0 ** -61), dict(ws=0), dict(ws=8),
    dict(score=1 << 20, seen=65), dict(reserved=1), dict(q=tensor(1 << 22), out=tensor(1 << 22))])
def test_attend_refuses(bad):
    assert attend(**bad) == EINVAL


def test_attend_refuses_a_small_workspace():
    need = kv.attend_workspace_bytes(1, 4, 128, 64, 4, 8)
    assert need > 0 and attend(ws_bytes=need - 1) == ENOSPC
    assert kv.lib().uzip_kv_attend(None, None, 1 << 25, 1 << 30, None) == EINVAL


@pytest.mark.parametrize("bad", [(0, 1, 8, 1, 1, 1), (1, 0, 8, 1, 1, 1), (1, 1, 4, 1, 1, 1), (1, 1, 8, 0, 1, 1), (1, 1, 8, 1, 0, 1),
                                 (1, 2, 8, 1, 1, 3), (1, 2, 8, 1, 1, 1), (65536, 1, 8, 1, 1, 1)])
def test_workspace_of_bad_shapes_is_zero(bad):
    assert kv.attend_workspace_bytes(*bad) == 0


def test_workspace_stays_small():
    """Partial results of split rows: within twice the cache's own size for single tokens, whatever the capacity."""
    for S in (1, 100, 2048, 131072, 1 << 20):
        for B in (1, 4, 32):
            assert kv.attend_workspace_bytes(B, 8, 128, S, 1, 64) <= 2 * B * S * 8 * 128 * 2 * 2 + (1 << 16)
    assert kv.evict_workspace_bytes(2, 8, 131072) > 0 and kv.evict_workspace_bytes(0, 8, 1) == 0


def append(c=None, q=None, out=None, k=None, v=None, length=1 << 24, drafted=0, dtype=0, T=4, heads=8, reserved=0, rope="good"):
    parts = [struct.unpack("=Q3q", t) for t in (q or tensor(), out or tensor(1 << 23), k or tensor(), v or tensor())]
    args = kv._APPEND.pack(*(x for p in parts for x in p), length, drafted, dtype, T, heads, reserved)
    return kv.lib().uzip_kv_append(c or cache(), args, rope_args() if rope == "good" else rope, None)


def rope_args(freq=1 << 20, pos=1 << 21, stride=4, rot=64, flags=0, amplitude=1.0, reserved=0):
    return kv._ROPE.pack(freq, pos, stride, rot, flags, amplitude, reserved)


BAD_ROPES = [dict(freq=0), dict(freq=4), dict(pos=2), dict(stride=-1), dict(rot=63), dict(rot=130), dict(flags=4), dict(amplitude=math.nan),
             dict(amplitude=math.inf), dict(reserved=1)]


@pytest.mark.parametrize("bad", BAD_ROPES)
def test_bad_ropes_are_refused(bad):
    assert append(rope=rope_args(**bad)) == EINVAL
    assert kv.lib().uzip_kv_rope(tensor(), tensor(1 << 23), 0, 1, 4, 8, 128, rope_args(**bad), None) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=tensor(0)), dict(out=tensor(0)), dict(out=tensor(1 << 22, (0, 2048, 128))), dict(k=tensor(0)), dict(v=tensor(12)),
    dict(length=0), dict(length=1), dict(drafted=1), dict(dtype=1), dict(dtype=2), dict(T=0), dict(heads=0), dict(reserved=1)])
def test_append_refuses(bad):
    assert append(**bad) == EINVAL


@pytest.mark.parametrize("args", [(None, tensor(), 0, 1, 4, 8, 128), (tensor(0), tensor(), 0, 1, 4, 8, 128), (tensor(), tensor(3), 0, 1, 4, 8, 128),
                                  (tensor(), tensor(1 << 23), 2, 1, 4, 8, 128), (tensor(), tensor(1 << 23), 0, 0, 4, 8, 128),
                                  (tensor(), tensor(1 << 23), 0, 1, 0, 8, 128), (tensor(), tensor(1 << 23), 0, 1, 4, 0, 128),
                                  (tensor(), tensor(1 << 23), 0, 1, 4, 8, 60), (tensor(), tensor(stride=(0, 2048, 128)), 0, 1, 4, 8, 128)])
def test_rope_refuses(args):
    assert kv.lib().uzip_kv_rope(*args, rope_args(), None) == EINVAL
    assert kv.lib().uzip_kv_rope(tensor(), tensor(1 << 23), 0, 1, 4, 8, 128, rope_args(pos=0), None) == EINVAL
    assert kv.lib().uzip_kv_rope(tensor(), tensor(1 << 23), 0, 1, 4, 8, 128, None, None) == EINVAL


def evict(c=None, out=None, score=1 << 24, ss=(256, 64), length=1 << 24, index=1 << 24, score_out=0, length_out=0, keep=16, sink=2,
          recent=4, seen=64, ws=1 << 25, ws_bytes=1 << 40):
    args = kv._EVICT.pack(score, *ss, length, index, score_out, length_out, keep, sink, recent, seen)
    return kv.lib().uzip_kv_evict(c or cache(), out or cache(k=1 << 26, v=1 << 27, tokens=16), args, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(out=cache(k=1 << 26, v=1 << 27, tokens=15)), dict(out=cache(k=1 << 26, v=1 << 27, tokens=16, heads=2)),
    dict(out=cache(k=1 << 26, v=1 << 27, tokens=16, dim=64)), dict(out=cache(k=1 << 26, v=1 << 27, tokens=16, dtype=1)),
    dict(out=cache(k=1 << 26, v=1 << 27, tokens=16, seqs=2)), dict(out=cache(tokens=16)),
    dict(out=cache(k=1 << 26, v=1 << 27, tokens=16, table=1 << 24, page=16, pages=4)), dict(score=0), dict(score=2), dict(ss=(-1, 0)),
    dict(length=0), dict(index=0), dict(index=2), dict(score_out=2), dict(length_out=1), dict(keep=0), dict(sink=17), dict(sink=10, recent=7),
    dict(seen=0), dict(seen=65), dict(ws=4), dict(c=cache(tokens=40000), seen=40000, ws=0)])
def test_evict_refuses(bad):
    assert evict(**bad) == EINVAL


def test_evict_refuses_a_small_workspace():
    assert kv.evict_workspace_bytes(1, 4, 32768) == 0
    assert evict(cache(tokens=40000), seen=40000, ws_bytes=kv.evict_workspace_bytes(1, 4, 40000) - 1) == ENOSPC


def test_structures_have_the_headers_sizes():
    """The packed layouts against the C compiler's."""
    import shutil
    import subprocess
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    names = {"uzip_kv_cache_t": kv._CACHE, "uzip_kv_rope_t": kv._ROPE, "uzip_kv_tensor_t": kv._TENSOR, "uzip_kv_append_args_t": kv._APPEND,
             "uzip_kv_attend_args_t": kv._ATTEND, "uzip_kv_evict_args_t": kv._EVICT}
    src = '#include "uzip_kv.h"\n' + "".join(f'_Static_assert(sizeof({n}) == {s.size}, "{n}");\n' for n, s in names.items())
    r = subprocess.run([cc, "-fsyntax-only", "-xc", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-"],
                       input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def test_host_tensors_and_wrong_shapes_are_refused():
    k = torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        kv.attend(q, k, k, n)
    with pytest.raises(ValueError, match="device tensors"):
        kv.evict(k, k, torch.zeros(2, 2, 8), n, 4)
    with pytest.raises(ValueError, match="device tensors"):
        kv.rope(q, torch.zeros(1, dtype=torch.int32), kv.rope_freq(64))
    with pytest.raises(ValueError, match="differ"):
        kv.attend(q, k, k[:, :4], n)
    with pytest.raises(ValueError, match="query heads"):
        kv.attend(torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16), k, k, n)
    with pytest.raises(ValueError, match="does not go with"):
        kv.attend(q.half(), k, k, n)
    with pytest.raises(ValueError, match="expected bfloat16"):
        kv.attend(q.float(), k, k, n)
    with pytest.raises(ValueError, match="not contiguous"):
        kv.attend(q, k.transpose(2, 3).contiguous().transpose(2, 3), k, n)
    with pytest.raises(ValueError, match="tree"):
        kv.attend(q, k, k, n, tree=torch.ones(2, 2, dtype=torch.bool))
    with pytest.raises(ValueError, match="table"):
        kv.attend(q, k, k, n, table=torch.zeros(2, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="sink"):
        kv.evict(k, k, torch.zeros(2, 2, 8), n, 4, sink=3, recent=2)
    with pytest.raises(ValueError, match="share memory"):
        kv.append(None, q[:, :, :2], q[:, :, :2], k[:1].expand(2, 8, 2, 64), k, n)
    with pytest.raises(ValueError, match="freq"):
        kv.rope(q, torch.zeros(1, dtype=torch.int32), torch.zeros(8))


def test_rope_freq():
    f = kv.rope_freq(8, 100.0)
    assert torch.allclose(f * 2 * math.pi, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(kv.rope_freq(8, 100.0, linear=4.0), f / 4.0)
    g = kv.rope_freq(8, 100.0, ntk=16.0)
    assert g[0] == f[0] and math.isclose(float(g[-1]), float(f[-1]) / 16.0, rel_tol=1e-14)
    # 1, 0.3.., 0.1, 0.03.. rad a position: turns over 100 positions 15.9, 5.03, 1.59, 0.503
    b = kv.rope_freq(8, 100.0, bands=(8.0, 100, 1.0, 4.0))
    assert torch.equal(b[:2], f[:2]) and b[3] == f[3] / 8.0
    keep = (float(f[2]) * 100 - 1.0) / 3.0
    assert math.isclose(float(b[2]), float(f[2]) * (keep + (1 - keep) / 8.0), rel_tol=1e-14)
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, base=-1.0), dict(rot=8, linear=0.0), dict(rot=2, ntk=2.0), dict(rot=8, bands=(0.0, 1, 1, 2)),
                dict(rot=8, bands=(2.0, 1, 2, 2))):
        with pytest.raises(ValueError):
            kv.rope_freq(**bad)


def test_errors_have_the_codecs_type():
    with pytest.raises(uzip.UzipError):
        kv._check(-1, "attend")
    assert ctypes.sizeof(ctypes.c_void_p) == 8
