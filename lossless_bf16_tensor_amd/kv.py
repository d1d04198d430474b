"""KV-cache operators (C-ABI: include/uzip_kv.h) over torch tensors.

What a serving step does to a cache before it is encoded for its transfer and
after it is decoded: :func:`rope`, :func:`append`, :func:`attend` and
:func:`evict`. Every step runs in the library's HIP kernels; this module checks
shapes, which the library cannot see, and passes pointers on.

Caches. ``k`` and ``v`` are [sequences, tokens, kv heads, head dim], or with a
page ``table`` (int32 [sequences, entries]) pools [pages, page, kv heads, head
dim]; page is a power of two, at least 16. They, queries and outputs may be any
views that start on a 16-byte boundary, whose last dim is contiguous and whose
other strides are multiples of 8 (that between tokens below 2^26), so a cache
kept [sequences, kv heads, tokens, head dim] is passed transposed. Element
types: bfloat16, float16, or float8_e5m2 beside queries of either. The head dim
is a multiple of 8 up to 256. No tensor is empty.

``length`` (int32 [sequences], on the device) counts the tokens each sequence
has; ``drafted`` (int32, optional) the new ones, when they are fewer than the
tensors hold. Values on the device are not checked, and none of them makes a
kernel read or write outside the tensors: lengths are clamped, table entries
outside the pool are absent pages.

Calls run on the current stream of the tensors' device, or on ``stream=``, and
can be captured. A workspace passed as ``ws=`` must not be shared by calls that
may overlap.

No gradient is recorded: tensors that require one are refused unless gradients
are switched off (``torch.no_grad``). :func:`rope` with ``inverse`` is the
gradient of :func:`rope`; the others serve inference.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

import torch

from .uzip import UzipError, lib as _codec_lib

# every symbol include/uzip_kv.h declares
EXPORTS = ("uzip_kv_rope", "uzip_kv_append", "uzip_kv_attend", "uzip_kv_attend_workspace_bytes", "uzip_kv_evict",
           "uzip_kv_evict_workspace_bytes")

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e5m2: 2}
_INTERLEAVED, _INVERSE = 1, 2

# uzip_kv_cache_t, uzip_kv_rope_t, uzip_kv_append_args_t, uzip_kv_attend_args_t, uzip_kv_evict_args_t
_CACHE = struct.Struct("=3Q7q8I")
_ROPE = struct.Struct("=2Qq2IfI")
_TENSOR = struct.Struct("=Q3q")
_APPEND = struct.Struct("=16q2Q4I")
_ATTEND = struct.Struct("=8q2Q2q3Q2q3If2I")
_EVICT = struct.Struct("=Q2q4Q4I")

_lib = None


def lib():
    """The library with the signatures of uzip_kv.h."""
    global _lib
    if _lib is None:
        L = _codec_lib()
        vp, u64, u32, st = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_char_p
        sig = {
            "uzip_kv_rope": (ctypes.c_int, [st, st, u32, u32, u32, u32, u32, st, vp]),
            "uzip_kv_append": (ctypes.c_int, [st, st, st, vp]),
            "uzip_kv_attend": (ctypes.c_int, [st, st, vp, u64, vp]),
            "uzip_kv_attend_workspace_bytes": (u64, [u32] * 6),
            "uzip_kv_evict": (ctypes.c_int, [st, st, st, vp, u64, vp]),
            "uzip_kv_evict_workspace_bytes": (u64, [u32] * 3),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


_EINVAL = -1


def _check(rc: int, what: str, **tensors):
    """Raises for a refusal; one of these tensors may be the reason. What the
    library checks is looked at here only then: a look at each tensor of a
    call takes longer than the smallest kernels."""
    if rc != 0:
        if rc == _EINVAL:
            for name, t in tensors.items():
                if t is not None:
                    _fits(t, name)
        raise UzipError(rc, f"{what}: {lib().uzip_strerror(rc).decode()}")


def _fits(t: torch.Tensor, what: str):
    """Raises with the reason why the library takes no such tensor [sequences, tokens, heads, head dim]."""
    if not t.numel():
        raise ValueError(f"{what} is empty: {tuple(t.shape)}")
    if t.shape[3] % 8 or t.shape[3] > 256:
        raise ValueError(f"{what}: the head dim is a multiple of 8 up to 256, got {t.shape[3]}")
    if t.data_ptr() % 16:
        raise ValueError(f"{what} does not start on a 16-byte boundary")
    st = _strides(t)
    if any(s % 8 for s in st):
        raise ValueError(f"{what}: strides are multiples of 8, got {t.stride()}")
    if st[1] >= 1 << 26:
        raise ValueError(f"{what}: the stride between tokens is below 2^26, got {st[1]}")


class _Here:
    """The current device and stream."""

    def __enter__(self):
        return self

    def __exit__(self, *e):
        return None


_HERE = _Here()


def _on(device: torch.device, stream):
    """A context that makes the tensors' device and `stream` (None: that
    device's current one) current, so that new tensors belong to it. The usual
    call, on the current device and stream, changes nothing: switching takes
    longer than the smallest kernels here."""
    if device.type != "cuda":
        raise ValueError("expected device tensors")
    if stream is not None:
        if stream.device != device:
            raise ValueError("the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return _HERE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _no_gradient():
    if torch.is_grad_enabled():
        raise ValueError("these operators record no gradient: call them under torch.no_grad(), or pass detached tensors "
                         "(the gradient of rope is rope with inverse=True)")


def _strides(t: torch.Tensor):
    """Strides of the first three dims; 0 for a dim of one element where its own does not fit the library's rules."""
    st = t.stride()
    if len(st) != 4:
        raise ValueError(f"expected four dims, got {len(st)}")
    s0, s1, s2, s3 = st
    if s3 != 1 and t.shape[3] != 1:
        raise ValueError("the head dim is not contiguous")
    if (s0 | s1 | s2) & 7 or s1 >= 1 << 26:
        return tuple(0 if t.shape[i] == 1 else st[i] for i in range(3))
    return s0, s1, s2


def _written(t: torch.Tensor, what: str):
    if 0 in t.stride():
        for n, s in zip(t.shape, t.stride()):
            if n != 1 and s == 0:
                raise ValueError(f"{what} has elements that share memory")


def _counts(t, seqs: int, device, what: str) -> int:
    """Address of an int32 tensor with one value a sequence; 0 for None."""
    if t is None:
        return 0
    if not (t.dtype == torch.int32 and t.shape == (seqs,) and t.is_contiguous() and t.device == device):
        raise ValueError(f"{what}: expected a contiguous int32 tensor of {seqs} on {device}")
    return t.data_ptr()


def _cache(k: torch.Tensor, v: torch.Tensor, table, seqs: int):
    """(packed uzip_kv_cache_t, kv heads, head dim, tokens a sequence)"""
    if not (k.shape == v.shape and k.dtype == v.dtype and k.device == v.device):
        raise ValueError("k and v caches differ in shape, type or device")
    dtype = _DTYPE.get(k.dtype)
    if dtype is None:
        raise ValueError(f"caches are bfloat16, float16 or float8_e5m2, got {k.dtype}")
    ks, vs = _strides(k), _strides(v)
    first, second, heads, dim = k.shape
    if table is None:
        if first != seqs:
            raise ValueError(f"the cache holds {first} sequences, expected {seqs}")
        return _CACHE.pack(k.data_ptr(), v.data_ptr(), 0, *ks, *vs, 0, dtype, seqs, heads, dim, second, 0, 0, 0), heads, dim, second
    if not (table.dtype == torch.int32 and table.dim() == 2 and table.shape[0] == seqs and table.device == k.device
            and table.shape[1] >= 1 and (table.stride(1) == 1 or table.shape[1] == 1)):
        raise ValueError(f"table: expected int32 [{seqs}, entries] with contiguous rows on {k.device}")
    if second < 16 or second & (second - 1):
        raise ValueError(f"pages hold a power of two of tokens, at least 16, got {second}")
    tokens = table.shape[1] * second
    return (_CACHE.pack(k.data_ptr(), v.data_ptr(), table.data_ptr(), *ks, *vs, table.stride(0) if seqs > 1 else 0, dtype,
                        seqs, heads, dim, tokens, second, first, 0), heads, dim, tokens)


def _score(score, seqs: int, heads: int, tokens: int, table, device):
    """((sequence, head) strides, tokens) of accumulated weights: as many tokens as the cache, or fewer when it is in pages."""
    n = score.shape[-1]
    if not (score.dtype == torch.float32 and score.shape == (seqs, heads, n) and score.device == device
            and (n == tokens or (table is not None and 1 <= n < tokens)) and (score.stride(2) == 1 or n == 1)):
        raise ValueError(f"score: expected float32 [{seqs}, {heads}, {tokens}] with contiguous rows on {device}")
    return score.stride()[:2], n


def _types(new: torch.Tensor, cache: torch.Tensor):
    if new.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {new.dtype}")
    if cache.dtype not in (new.dtype, torch.float8_e5m2):
        raise ValueError(f"{new.dtype} does not go with a {cache.dtype} cache")


def _rope(freq, pos, amplitude: float, flags: int, seqs: int, tokens: int, dim: int, device):
    """Packed uzip_kv_rope_t."""
    if not (freq.dtype == torch.float64 and freq.dim() == 1 and freq.is_contiguous() and freq.device == device):
        raise ValueError(f"freq: expected a contiguous float64 vector on {device}")
    if 2 * freq.numel() > dim:
        raise ValueError(f"freq turns {2 * freq.numel()} of {dim} elements")
    at = stride = 0
    if pos is not None:
        if not (pos.dtype == torch.int32 and pos.device == device and pos.shape in ((seqs, tokens), (tokens,))
                and (pos.stride(-1) == 1 or tokens == 1)):
            raise ValueError(f"pos: expected int32 [{seqs}, {tokens}] or [{tokens}] with contiguous rows on {device}")
        at, stride = pos.data_ptr(), pos.stride(0) if pos.dim() == 2 and seqs > 1 else 0
    return _ROPE.pack(freq.data_ptr(), at, stride, 2 * freq.numel(), flags, amplitude, 0)


def rope_freq(rot: int, base: float = 10000.0, *, linear: float = 1.0, ntk: float = 1.0, bands=None,
              device=None) -> torch.Tensor:
    """Turns per position of the rot / 2 pairs of a rotary embedding, float64:
    base ** (-2 i / rot) / (2 pi), scaled for contexts longer than trained on.

    linear: all positions divided by this factor.
    ntk:    base times factor ** (rot / (rot - 2)), which slows the slowest
            pair by the factor and leaves the fastest.
    bands:  (factor, trained, low, high): pairs that turn at most `low` times
            over the `trained` positions are slowed by the factor, those that
            turn at least `high` times are kept, and between them the two
            frequencies are mixed in proportion.
    """
    if not (rot >= 2 and rot % 2 == 0):
        raise ValueError(f"rot is even and positive, got {rot}")
    if not (base > 0 and linear > 0 and ntk > 0):
        raise ValueError("base and factors are positive")
    if ntk != 1.0:
        if rot <= 2:
            raise ValueError("ntk scaling needs more than one pair")
        base = base * ntk ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot) / (2.0 * math.pi) / linear
    if bands is not None:
        factor, trained, low, high = bands
        if not (factor > 0 and high > low):
            raise ValueError("bands: expected a positive factor and low < high")
        keep = ((f * trained - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f if device is None else f.to(device)


def rope(x: torch.Tensor, pos: torch.Tensor, freq: torch.Tensor, *, amplitude: float = 1.0, interleaved: bool = False,
         inverse: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x [sequences, tokens, heads, dim], bfloat16 or
    float16. pos: int32 [sequences, tokens] or [tokens]. freq: turns per
    position of each pair (:func:`rope_freq`); the first 2 * len(freq) elements
    turn, as halves (i, i + len(freq)) or interleaved (2i, 2i + 1). inverse
    turns back: the gradient, and what moves kept keys to other positions. out
    may be x."""
    if x.requires_grad or freq.requires_grad or (out is not None and out.requires_grad):
        _no_gradient()
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"expected bfloat16 or float16, got {x.dtype}")
    xs = _strides(x)
    B, T, H, D = x.shape
    dev = x.device
    packed = _rope(freq, pos, amplitude, interleaved * _INTERLEAVED | inverse * _INVERSE, B, T, D, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((B, T, H, D), dtype=x.dtype, device=dev)
        else:
            if not (out.shape == x.shape and out.dtype == x.dtype and out.device == dev):
                raise ValueError("out differs from x in shape, type or device")
            _written(out, "out")
        rc = lib().uzip_kv_rope(_TENSOR.pack(x.data_ptr(), *xs), _TENSOR.pack(out.data_ptr(), *_strides(out)),
                                _DTYPE[x.dtype], B, T, H, D, packed, _stream(dev))
    if rc:
        _check(rc, "rope", x=x, out=out)
    return out


def append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           length: torch.Tensor, freq: torch.Tensor | None = None, *, pos: torch.Tensor | None = None,
           table: torch.Tensor | None = None, drafted: torch.Tensor | None = None, amplitude: float = 1.0,
           interleaved: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Writes new tokens' keys k (turned to their positions) and values v
    [sequences, tokens, kv heads, dim] into the cache behind each sequence's
    length tokens, and returns the turned queries q [sequences, tokens, heads,
    dim]; q may be None. pos defaults to length + 0, 1, ...; without freq
    nothing turns. length is not changed. Tokens from drafted on, past the
    cache's end or in an absent page are not written. out may be q; nothing else
    that is written may overlap another tensor."""
    if (k.requires_grad or v.requires_grad or k_cache.requires_grad or v_cache.requires_grad or (q is not None and q.requires_grad)
            or (freq is not None and freq.requires_grad) or (out is not None and out.requires_grad)):
        _no_gradient()
    B, T, H, D = k.shape
    if not (v.shape == k.shape and v.dtype == k.dtype and v.device == k.device):
        raise ValueError("k and v differ in shape, type or device")
    _types(k, k_cache)
    cache, heads, dim, _ = _cache(k_cache, v_cache, table, B)
    _written(k_cache, "the key cache")
    _written(v_cache, "the value cache")
    dev = k.device
    if k_cache.device != dev:
        raise ValueError("the cache is on another device")
    if not (heads == H and dim == D):
        raise ValueError(f"the cache has {heads} heads of {dim}, the new keys {H} of {D}")
    packed = None
    if freq is not None:
        packed = _rope(freq, pos, amplitude, interleaved * _INTERLEAVED, B, T, D, dev)
    with _on(dev, stream):
        if q is None:
            qs = (0,) * 8
            hq = 0
        else:
            if not (q.dim() == 4 and q.shape[0] == B and q.shape[1] == T and q.shape[3] == D and q.dtype == k.dtype
                    and q.device == dev):
                raise ValueError("q does not go with k")
            hq = q.shape[2]
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            else:
                if not (out.shape == q.shape and out.dtype == q.dtype and out.device == dev):
                    raise ValueError("out differs from q in shape, type or device")
                _written(out, "out")
            qs = (q.data_ptr(), *_strides(q), out.data_ptr(), *_strides(out))
        args = _APPEND.pack(*qs, k.data_ptr(), *_strides(k), v.data_ptr(), *_strides(v), _counts(length, B, dev, "length"),
                            _counts(drafted, B, dev, "drafted"), _DTYPE[k.dtype], T, hq, 0)
        rc = lib().uzip_kv_append(cache, args, packed, _stream(dev))
    if rc:
        _check(rc, "append", q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, out=out)
    return out if q is not None else None


@functools.lru_cache(maxsize=4096)
def attend_workspace_bytes(seqs: int, kv_heads: int, dim: int, cache_tokens: int, tokens: int, heads: int) -> int:
    """Workspace that :func:`attend` needs for these shapes; 0 when they are invalid."""
    return int(lib().uzip_kv_attend_workspace_bytes(seqs, kv_heads, dim, cache_tokens, tokens, heads))


def attend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, length: torch.Tensor, *,
           table: torch.Tensor | None = None, tree: torch.Tensor | None = None, drafted: torch.Tensor | None = None,
           scale: float | None = None, score: torch.Tensor | None = None, lse: torch.Tensor | None = None,
           out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the drafted tokens q [sequences, tokens, heads, dim] over a
    cache that holds length earlier tokens and, behind them, the drafted ones'
    keys and values (:func:`append`). A drafted token sees every earlier token
    and those drafted ones that its row of tree (bool [tokens, tokens], or one
    such per sequence) names; without a tree, those up to itself. heads is a
    multiple of the cache's. scale defaults to 1 / sqrt(dim).

    score (float32 [sequences, kv heads, cache tokens]) has the weight that each
    cached token received from the drafted tokens and the heads that share it
    added. A cache in pages may end behind the last token of score: what is
    there is not added. lse (float32 [sequences, tokens, heads], contiguous) receives the log
    of each query's sum of exponentials. A query that sees nothing gives zeros
    and -inf, as do those from drafted on. Masked keys and values have no
    effect, whatever they hold. out does not overlap the inputs."""
    if (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad or (score is not None and score.requires_grad)
            or (lse is not None and lse.requires_grad) or (out is not None and out.requires_grad)):
        _no_gradient()
    _types(q, k_cache)
    qs = _strides(q)
    B, T, hq, D = q.shape
    dev = q.device
    cache, heads, dim, tokens = _cache(k_cache, v_cache, table, B)
    if k_cache.device != dev:
        raise ValueError("the cache is on another device")
    if not (dim == D and hq >= heads > 0 and hq % heads == 0):
        raise ValueError(f"{hq} query heads of {D} do not go with {heads} heads of {dim}")
    ts = (0, 0)
    if tree is not None:
        if not (tree.dtype in (torch.bool, torch.uint8) and tree.device == dev and tree.shape in ((T, T), (B, T, T))
                and (tree.stride(-1) == 1 or T == 1)):
            raise ValueError(f"tree: expected bool [{T}, {T}] or [{B}, {T}, {T}] with contiguous rows on {dev}")
        ts = (tree.stride(0) if tree.dim() == 3 else 0, tree.stride(-2))
    ss, seen = (0, 0), 0
    if score is not None:
        ss, seen = _score(score, B, heads, tokens, table, dev)
        _written(score, "score")
    if lse is not None:
        if not (lse.dtype == torch.float32 and lse.shape == (B, T, hq) and lse.is_contiguous() and lse.device == dev):
            raise ValueError(f"lse: expected contiguous float32 [{B}, {T}, {hq}] on {dev}")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((B, T, hq, D), dtype=q.dtype, device=dev)
        else:
            if not (out.shape == q.shape and out.dtype == q.dtype and out.device == dev):
                raise ValueError("out differs from q in shape, type or device")
            _written(out, "out")
        if ws is None:
            ws = torch.empty(attend_workspace_bytes(B, heads, D, tokens, T, hq), dtype=torch.uint8, device=dev)
        else:
            if not (ws.dtype == torch.uint8 and ws.is_contiguous() and ws.device == dev):
                raise ValueError(f"ws: expected contiguous uint8 on {dev} from a 16-byte boundary")
        args = _ATTEND.pack(q.data_ptr(), *qs, out.data_ptr(), *_strides(out), lse.data_ptr() if lse is not None else 0,
                            score.data_ptr() if score is not None else 0, *ss, _counts(length, B, dev, "length"),
                            _counts(drafted, B, dev, "drafted"), tree.data_ptr() if tree is not None else 0, *ts,
                            _DTYPE[q.dtype], T, hq, 1.0 / math.sqrt(D) if scale is None else scale, seen, 0)
        rc = lib().uzip_kv_attend(cache, args, ws.data_ptr(), ws.numel(), _stream(dev))
    if rc:
        _check(rc, "attend", q=q, k_cache=k_cache, v_cache=v_cache, out=out)
    return out


@functools.lru_cache(maxsize=4096)
def evict_workspace_bytes(seqs: int, kv_heads: int, cache_tokens: int) -> int:
    """Workspace that :func:`evict` needs for scores of cache_tokens; 0 when it needs none or the shapes are invalid."""
    return int(lib().uzip_kv_evict_workspace_bytes(seqs, kv_heads, cache_tokens))


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, score: torch.Tensor, length: torch.Tensor, keep: int, *,
          sink: int = 0, recent: int = 0, table: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
          v_out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Cuts a cache to keep tokens per sequence and head: the first `sink`, the
    last `recent`, and the others with the largest score (float32 [sequences, kv
    heads, cache tokens], as :func:`attend` adds it up), ties to the lower
    token, NaN last. A cache in pages may have more tokens than score: it is taken to
    end with it. Returns (k, v, score, length, index): caches [sequences,
    keep, kv heads, dim] with the kept tokens in order and zeros behind them,
    ready for ``uzip.encode``; their scores [sequences, kv heads, keep]; min(length,
    keep); and where each came from, int32 [sequences, kv heads, keep], -1
    behind the last. Keys keep the positions they were turned to. Launches are
    sized by what score can hold, not by length: where caches are much larger
    than what is in them, pass slices that end behind the longest sequence."""
    if (k_cache.requires_grad or v_cache.requires_grad or score.requires_grad or (k_out is not None and k_out.requires_grad)
            or (v_out is not None and v_out.requires_grad)):
        _no_gradient()
    B = length.numel()
    cache, heads, dim, tokens = _cache(k_cache, v_cache, table, B)
    dev = k_cache.device
    ss, seen = _score(score, B, heads, tokens, table, dev)
    if not (1 <= keep <= 1 << 30 and sink >= 0 and recent >= 0 and sink + recent <= keep):
        raise ValueError(f"keep {keep}, sink {sink}, recent {recent}: expected 1 <= keep and sink + recent <= keep")
    with _on(dev, stream):
        made = []
        for t in (k_out, v_out):
            if t is None:
                t = torch.empty((B, keep, heads, dim), dtype=k_cache.dtype, device=dev)
            else:
                if not (t.shape == (B, keep, heads, dim) and t.dtype == k_cache.dtype and t.device == dev):
                    raise ValueError(f"k_out, v_out: expected {k_cache.dtype} [{B}, {keep}, {heads}, {dim}] on {dev}")
                _written(t, "k_out or v_out")
            made.append(t)
        kept, index = torch.empty((B, heads, keep), dtype=torch.float32, device=dev), torch.empty((B, heads, keep), dtype=torch.int32, device=dev)
        left = torch.empty(B, dtype=torch.int32, device=dev)
        if ws is None:
            need = evict_workspace_bytes(B, heads, seen)
            ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        elif not (ws.dtype == torch.uint8 and ws.is_contiguous() and ws.device == dev):
            raise ValueError(f"ws: expected contiguous uint8 on {dev} from a 16-byte boundary")
        args = _EVICT.pack(score.data_ptr(), *ss, _counts(length, B, dev, "length"),
                           index.data_ptr(), kept.data_ptr(), left.data_ptr(), keep, sink, recent, seen)
        rc = lib().uzip_kv_evict(cache, _cache(*made, None, B)[0], args, 0 if ws is None else ws.data_ptr(),
                                 0 if ws is None else ws.numel(), _stream(dev))
    if rc:
        _check(rc, "evict", k_cache=k_cache, v_cache=v_cache, k_out=made[0], v_out=made[1])
    return made[0], made[1], kept, left, index
