"""CPU tests of the host side of the operators of drafted tokens and of 8-bit
caches with scales: structures, sizes and refusals. Every call below returns
before it touches the GPU."""
import os
import shutil
import struct
import subprocess

import pytest
import torch

from lossless_bf16_tensor_amd import kv
from test_kv_host import BAD_CACHES, BAD_ROPES, EINVAL, ENOSPC, ROOT, cache, rope_args, tensor

BF16, E4M3, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8


def test_structures_have_the_headers_sizes():
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    names = {"uzip_kv_scales_t": kv._SCALES, "uzip_kv_verify_args_t": kv._VERIFY, "uzip_kv_accept_args_t": kv._ACCEPT,
             "uzip_kv_pages_t": kv._PAGES, "uzip_kv_pool_t": kv._POOL}
    src = '#include "uzip_kv.h"\n' + "".join(f'_Static_assert(sizeof({n}) == {s.size}, "{n}");\n' for n, s in names.items())
    r = subprocess.run([cc, "-fsyntax-only", "-xc", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-"],
                       input=src, text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def scales(k=1 << 26, v=1 << 27, ks=(0, 4, 1), vs=(0, 4, 1), block=16, reserved=0):
    return kv._SCALES.pack(k, v, *ks, *vs, block, reserved)


def attend(c=None, f=None, q=None, out=None, dtype=0, T=4, heads=8, scale=0.1, ws=1 << 25, ws_bytes=1 << 40):
    args = kv._ATTEND.pack(*struct.unpack("=Q3q", q or tensor()), *struct.unpack("=Q3q", out or tensor(1 << 21)), 0, 0, 256, 64, 1 << 24,
                           0, 0, 0, 4, dtype, T, heads, scale, 64, 0)
    return kv.lib().uzip_kv_attend_scaled(c or cache(dtype=4), scales() if f is None else f, args, ws, ws_bytes, None)


def append(c=None, f=None, q=None, out=None, k=None, v=None, length=1 << 24, dtype=0, T=4, heads=8, rope="good"):
    parts = [struct.unpack("=Q3q", t) for t in (q or tensor(), out or tensor(1 << 23), k or tensor(), v or tensor())]
    args = kv._APPEND.pack(*(x for p in parts for x in p), length, 0, dtype, T, heads, 0)
    return kv.lib().uzip_kv_append_scaled(c or cache(dtype=4), scales() if f is None else f, args, rope_args() if rope == "good" else rope, None)


@pytest.mark.parametrize("bad", [b for b in BAD_CACHES if "dtype" not in b] + [dict(dtype=d) for d in (0, 1, 2, 5)])
def test_bad_caches_are_refused(bad):
    c = cache(**{"dtype": 3, **bad})
    assert attend(c) == EINVAL and append(c) == EINVAL


@pytest.mark.parametrize("bad", [dict(k=0), dict(v=0), dict(k=2), dict(v=(1 << 27) + 1), dict(ks=(-1, 4, 1)), dict(vs=(0, -4, 1)), dict(vs=(0, 4, -1)),
                                 dict(block=0), dict(block=8), dict(block=24), dict(reserved=1), dict(ks=(1 << 41, 4, 1))])
def test_bad_scales_are_refused(bad):
    assert attend(f=scales(**bad)) == EINVAL and append(f=scales(**bad)) == EINVAL


def test_scales_are_no_wider_than_a_page():
    c = cache(dtype=4, table=1 << 23, page=32, pages=4, tokens=64)
    assert attend(c, scales(block=64)) == EINVAL and append(c, scales(block=64)) == EINVAL
    assert attend(c, scales(block=32), ws=0) == EINVAL


def test_other_refusals_of_caches_with_scales():
    assert kv.lib().uzip_kv_attend_scaled(cache(dtype=4), None, None, 1 << 25, 1 << 30, None) == EINVAL
    for bad in (dict(dtype=2), dict(T=0), dict(heads=6), dict(scale=0.0), dict(ws=0), dict(q=tensor(8)), dict(out=tensor(1 << 22))):
        assert attend(**bad) == EINVAL, bad
    assert attend(ws_bytes=kv.attend_workspace_bytes(1, 4, 128, 64, 4, 8, True) - 1) == ENOSPC
    for bad in (dict(dtype=2), dict(T=0), dict(heads=0), dict(length=0), dict(k=tensor(0)), dict(v=tensor(12)), dict(q=tensor(0)),
                dict(out=tensor(1 << 22, (0, 2048, 128))), dict(out=tensor(1 << 23), k=tensor(1 << 23)), dict(f=scales(v=1 << 26)),
                dict(c=cache(dtype=4, v=1 << 20))):
        assert append(**bad) == EINVAL, bad
    for bad in BAD_ROPES:
        assert append(rope=rope_args(**bad)) == EINVAL


def test_workspace_of_attention_over_scales():
    """Parts of split rows: within a few times the queries' own size in binary32, whatever the capacity; none for bad shapes."""
    assert kv.attend_workspace_bytes(0, 4, 128, 64, 4, 8, True) == kv.attend_workspace_bytes(1, 4, 128, 64, 4, 6, True) == 0
    for B in (1, 7, 64, 500):
        for T in (1, 5, 64):
            for S in (1, 100, 20000, 1 << 20):
                rows = B * T * 64
                parts = 1 + 4 * (2048 // B + 1)
                assert kv.attend_workspace_bytes(B, 8, 128, S, T, 64, True) <= rows * parts * 128 * 5 + (1 << 16)


def verify(target=1 << 20, draft=0, ps=(400, 100), qs=(400, 100), tokens=1 << 24, parent=0, drafted=0, uniform=1 << 24, tok=4, par=4, us=4,
           path=1 << 25, count=1 << 25, token=1 << 25, dtype=2, B=2, T=4, V=100, reserved=0, ws=1 << 26, ws_bytes=1 << 40):
    args = kv._VERIFY.pack(target, draft, *ps, *qs, tokens, parent, drafted, uniform, tok, par, us, path, count, token, dtype, B, T, V, reserved)
    return kv.lib().uzip_kv_verify(args, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(target=0), dict(target=2), dict(target=1, dtype=0), dict(draft=2), dict(ps=(-1, 100)), dict(ps=(400, -1)), dict(qs=(400, -1)),
    dict(ps=(1 << 41, 100)), dict(tokens=0), dict(tokens=2), dict(parent=2), dict(drafted=3), dict(uniform=0), dict(uniform=1), dict(tok=-1),
    dict(par=-1), dict(us=-1), dict(path=0), dict(path=2), dict(count=0), dict(token=0), dict(token=1), dict(dtype=3), dict(B=0), dict(B=65536),
    dict(T=0), dict(T=1025), dict(V=0), dict(V=(1 << 30) + 1), dict(reserved=1), dict(ws=0), dict(ws=8)])
def test_verify_refuses(bad):
    assert verify(**bad) == EINVAL


def test_verify_refuses_a_small_workspace():
    need = kv.verify_workspace_bytes(2, 4, 100)
    assert need > 0 and verify(ws_bytes=need - 1) == ENOSPC
    assert kv.verify_workspace_bytes(0, 4, 100) == kv.verify_workspace_bytes(2, 1025, 100) == kv.verify_workspace_bytes(2, 4, 0) == 0
    assert kv.lib().uzip_kv_verify(None, 1 << 26, 1 << 30, None) == EINVAL


def accept(c=None, length=1 << 24, path=1 << 24, stride=4, count=1 << 24, nodes=4, reserved=0):
    return kv.lib().uzip_kv_accept(c or cache(), kv._ACCEPT.pack(length, path, stride, count, nodes, reserved), None)


@pytest.mark.parametrize("bad", [dict(length=0), dict(length=2), dict(path=0), dict(path=2), dict(stride=-1), dict(count=0), dict(count=1),
                                 dict(nodes=0), dict(nodes=1025), dict(reserved=1)] + [dict(c=cache(**b)) for b in BAD_CACHES + [dict(v=1 << 20), dict(dtype=4)]])
def test_accept_refuses(bad):
    assert accept(**bad) == EINVAL


def pages(call="fork", table=1 << 20, stride=4, length=1 << 21, parent=1 << 21, held=0, out=1 << 22, out_length=1 << 23, moves=1 << 24,
          left=1 << 24, rows=2, seqs=3, entries=4, pages=10, page=16, room=1, reserved=0, ws=1 << 25, ws_bytes=1 << 40):
    args = kv._PAGES.pack(table, stride, length, parent, held, out, out_length, moves, left, rows, seqs, entries, pages, page, room, reserved)
    return getattr(kv.lib(), "uzip_kv_" + call)(args, ws, ws_bytes, None)


BAD_PAGES = [dict(table=0), dict(table=2), dict(stride=-1), dict(length=0), dict(length=2), dict(out=0), dict(out=2), dict(moves=0), dict(moves=1), dict(left=0),
             dict(rows=0), dict(rows=65536), dict(seqs=0), dict(seqs=65536), dict(entries=0), dict(pages=0), dict(pages=(1 << 30) + 1), dict(page=8),
             dict(page=24), dict(page=1 << 29, entries=4), dict(reserved=1), dict(ws=0), dict(ws=4), dict(out=1 << 20)]


@pytest.mark.parametrize("bad", BAD_PAGES + [dict(parent=0), dict(parent=2), dict(out_length=0), dict(out_length=1), dict(out_length=1 << 21), dict(room=(1 << 30) + 1)])
def test_fork_refuses(bad):
    assert pages(**bad) == EINVAL


COMPACT = dict(call="compact", parent=0, out_length=0, room=0, rows=3)


@pytest.mark.parametrize("bad", [b for b in BAD_PAGES] + [dict(parent=1 << 21), dict(out_length=1 << 23), dict(room=1), dict(rows=2)])
def test_compact_refuses(bad):
    assert pages(**{**COMPACT, **bad}) == EINVAL


def test_small_workspaces_of_pages():
    need = kv.pages_workspace_bytes(10, 3, 4)
    assert need > 0 and pages(ws_bytes=need - 1) == ENOSPC and pages(**COMPACT, ws_bytes=need - 1) == ENOSPC
    assert kv.pages_workspace_bytes(0, 3, 4) == kv.pages_workspace_bytes(10, 0, 4) == kv.pages_workspace_bytes(10, 3, 0) == 0
    assert kv.lib().uzip_kv_fork(None, 1 << 25, 1 << 30, None) == EINVAL


def pool(data=1 << 20, page=4096, s=(256, 16), n=(4, 4), run=16, reserved=0):
    return kv._POOL.pack(data, page, *s, *n, run, reserved)


@pytest.mark.parametrize("bad", [dict(data=0), dict(page=-1), dict(s=(-1, 16)), dict(s=(256, -16)), dict(n=(0, 4)), dict(n=(4, 0)), dict(run=0), dict(run=(1 << 30) + 1),
                                 dict(n=(1 << 20, 1 << 20)), dict(reserved=1)])
def test_copy_pages_refuses(bad):
    f = kv.lib().uzip_kv_copy_pages
    assert f(1 << 22, 4, pool(**bad), 1, 10, None) == EINVAL
    assert f(1 << 22, 4, pool() + pool(**bad), 2, 10, None) == EINVAL


def test_copy_pages_refuses_more():
    f = kv.lib().uzip_kv_copy_pages
    for args in ((0, 4, pool(), 1, 10), (2, 4, pool(), 1, 10), (1 << 22, (1 << 30) + 1, pool(), 1, 10), (1 << 22, 4, None, 1, 10), (1 << 22, 4, pool(), 0, 10),
                 (1 << 22, 4, pool() * 9, 9, 10), (1 << 22, 4, pool(), 1, 0)):
        assert f(*args, None) == EINVAL, args
    assert f(1 << 22, 0, pool(), 1, 10, None) == 0          # nothing to copy


def test_pools_as_runs():
    """Any order of dims, merged where they follow each other."""
    for t, want in ((torch.zeros(5, 16, 4, 32, dtype=BF16), (4096, 0, 0, 1, 1, 4096)),
                    (torch.zeros(5, 4, 16, 32, dtype=BF16).transpose(1, 2), (4096, 0, 0, 1, 1, 4096)),
                    (torch.zeros(5, 16, 8, 32, dtype=BF16)[:, :, 2:6], (8192, 0, 512, 1, 16, 256)),
                    (torch.zeros(5, 16, 8, 64, dtype=BF16)[:, :, 2:6, :32], (16384, 1024, 128, 16, 4, 64)),
                    (torch.zeros(5, 2, 8), (64, 0, 0, 1, 1, 64)), (torch.zeros(1, 16, dtype=I8), (0, 0, 0, 1, 1, 16))):
        assert kv._pool(t.shape, t.stride(), t.element_size()) == want
    with pytest.raises(ValueError, match="two dims"):
        t = torch.zeros(5, 4, 6, 8, 10)[:, ::2, ::2, ::2, ::2]
        kv._pool(t.shape, t.stride(), 4)


@pytest.mark.parametrize("tokens,blocks,block", [(16, 1, 16), (17, 2, 16), (17, 1, 32), (100, 7, 16), (100, 4, 32), (100, 2, 64), (100, 1, 128), (64, 4, 16),
                                                 (1, 1, 16), (131072, 2048, 64), (100, 3, 0), (100, 8, 0), (100, 0, 0), (131072, 1, 0)])
def test_block_by_the_number_of_scales(tokens, blocks, block):
    assert kv._block((1, blocks, 1), (1, tokens, 1, 64)) == block


def operands(dtype=E4M3):
    k, v = torch.zeros(2, 32, 2, 64, dtype=dtype), torch.zeros(2, 32, 2, 64, dtype=dtype)
    q, new = torch.zeros(2, 1, 4, 64, dtype=BF16), torch.zeros(2, 1, 2, 64, dtype=BF16)
    return dict(k=k, v=v, ks=torch.ones(2, 2, 2), vs=torch.ones(2, 2, 2), n=torch.zeros(2, dtype=torch.int32), q=q, new=new, new_v=new.clone(),
                p=torch.ones(2, 3, 10), d=torch.ones(2, 3, 10), tok=torch.zeros(2, 3, dtype=torch.int32), u=torch.zeros(2, 3),
                k16=torch.zeros(2, 32, 2, 64, dtype=BF16), v16=torch.zeros(2, 32, 2, 64, dtype=BF16), path=torch.zeros(2, 3, dtype=torch.int32),
                table=torch.zeros(2, 3, dtype=torch.int32), pool=torch.zeros(4, 16, 2), moves=torch.zeros(2, 2, dtype=torch.int32))


CALLS = dict(append=lambda o: kv.append(o["q"], o["new"], o["new_v"], o["k"], o["v"], o["n"], k_scale=o["ks"], v_scale=o["vs"]),
             attend=lambda o: kv.attend(o["q"], o["k"], o["v"], o["n"], k_scale=o["ks"], v_scale=o["vs"]),
             verify=lambda o: kv.verify(o["tok"], o["p"], o["u"], draft=o["d"]),
             accept=lambda o: kv.accept(o["k16"], o["v16"], o["n"], o["path"], o["n"]),
             fork=lambda o: kv.fork(o["table"], o["n"], o["n"], 4, 16),
             compact=lambda o: kv.compact(o["table"], o["n"], 4, 16),
             copy=lambda o: kv.copy_pages(o["moves"], o["pool"]))


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="device tensors"):
        CALLS[call](operands())


@pytest.mark.parametrize("call,names", [("append", ("q", "new", "new_v", "ks", "vs")), ("attend", ("q", "ks", "vs")), ("verify", ("p", "d", "u")),
                                        ("accept", ("k16", "v16")), ("copy", ("pool",))])
def test_tensors_that_require_a_gradient(call, names):
    for name in names:
        o = operands()
        o[name].requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            CALLS[call](o)
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            CALLS[call](o)


def test_scales_that_do_not_fit():
    for name, t in (("ks", None), ("vs", None), ("ks", torch.ones(2, 3, 2)), ("vs", torch.ones(2, 1, 2)), ("ks", torch.ones(2, 2, 1)),
                    ("ks", torch.ones(2, 2, 2, dtype=torch.float64)), ("vs", torch.ones(2, 2)), ("ks", torch.ones(1, 2, 2))):
        for call in ("append", "attend"):
            with pytest.raises(ValueError, match="k_scale"):
                CALLS[call](dict(operands(), **{name: t}))
    o = operands()
    with pytest.raises(ValueError, match="share memory"):
        CALLS["append"](dict(o, ks=torch.ones(2, 2, 1).expand(2, 2, 2)))
    for call in ("append", "attend"):                 # scales beside a cache that has none, and none beside one that does
        with pytest.raises(ValueError, match="with scales float8_e4m3fn or int8"):
            CALLS[call](dict(o, k=o["k16"], v=o["v16"]))
        with pytest.raises(ValueError, match="go with k_scale"):
            CALLS[call](dict(o, ks=None, vs=None))
    with pytest.raises(ValueError, match="go with k_scale"):
        kv.accept(o["k"], o["v"], o["n"], o["path"], o["n"])
    with pytest.raises(ValueError, match="go with k_scale"):
        kv.evict(o["k"], o["v"], torch.zeros(2, 2, 32), o["n"], 4)


@pytest.mark.parametrize("change,why", [
    (dict(p=torch.ones(2, 3, 10, dtype=torch.float64)), "float32, bfloat16"), (dict(d=torch.ones(2, 3, 9)), "draft differs"),
    (dict(d=torch.ones(2, 3, 10, dtype=BF16)), "draft differs"), (dict(tok=torch.zeros(2, 3, dtype=torch.int64)), "tokens"),
    (dict(tok=torch.zeros(2, 2, dtype=torch.int32)), "tokens"), (dict(u=torch.zeros(2, 3, dtype=torch.float64)), "uniform"),
    (dict(p=torch.ones(2, 10)), "vocabulary"), (dict(p=torch.ones(2, 10, 3).transpose(1, 2)), "not contiguous"), (dict(p=torch.ones(2, 0, 10)), "vocabulary")])
def test_probabilities_that_do_not_fit(change, why):
    with pytest.raises(ValueError, match=why):
        CALLS["verify"](dict(operands(), **change))


def test_trees_that_do_not_fit():
    o = operands()
    for parent in (torch.zeros(4, dtype=torch.int32), torch.zeros(3, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError, match="parent"):
            kv.verify(o["tok"], o["p"], o["u"], parent=parent)
    with pytest.raises(ValueError, match="1024"):
        kv.verify(torch.zeros(1, 1025, dtype=torch.int32), torch.ones(1, 1025, 2), torch.zeros(1, 1025))
    with pytest.raises(ValueError, match="path"):
        kv.accept(o["k16"], o["v16"], o["n"], torch.zeros(2, 1025, dtype=torch.int32), o["n"])
    with pytest.raises(ValueError, match="path"):
        kv.accept(o["k16"], o["v16"], o["n"], torch.zeros(3, 3, dtype=torch.int32), o["n"])


def test_tables_that_do_not_fit():
    o = operands()
    for table, pages_, page, kw, why in ((o["table"].long(), 4, 16, {}, "table"), (o["table"][:, :0], 4, 16, {}, "table"), (o["table"], 4, 8, {}, "power of two"),
                                         (o["table"], 4, 24, {}, "power of two"), (o["table"], 0, 16, {}, "pages"), (o["table"], 4, 16, dict(room=-1), "room"),
                                         (o["table"], 4, 16, dict(held=torch.zeros(3, dtype=torch.bool)), "held")):
        with pytest.raises(ValueError, match=why):
            kv.fork(table, o["n"], o["n"], pages_, page, **kw)
    with pytest.raises(ValueError, match="no sequences"):
        kv.fork(o["table"], o["n"], o["n"][:0], 4, 16)
    with pytest.raises(ValueError, match="held"):
        kv.compact(o["table"], o["n"], 4, 16, held=torch.zeros(3, dtype=torch.bool))


def test_pools_that_do_not_fit():
    o = operands()
    for pools, why in (((), "1 to 8"), ((o["pool"],) * 9, "1 to 8"), ((o["pool"], o["pool"][:3]), "as many pages"), ((o["pool"][:, :0],), "pages"),
                       ((torch.zeros(4),), "pages"), ((torch.zeros(1, 16, 2).expand(4, 16, 2),), "share memory")):
        with pytest.raises(ValueError, match=why):
            kv.copy_pages(o["moves"], *pools)
    for moves in (o["moves"].long(), o["moves"][:, :1], o["moves"].t()[:, :1].expand(2, 2)):
        with pytest.raises(ValueError, match="moves"):
            kv.copy_pages(moves, o["pool"])
