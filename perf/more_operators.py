"""Cases of the operators of a serving step with drafted tokens over 8-bit caches in pages.

A server that answers with a transferred KV cache keeps it in 8 bits with a
scale for each block of tokens and head, in pages that its sequences share, and
lets a small model draft the tokens that the large one then checks. Measured
here, next to the operators of perf/operators.py:

  append   new tokens' keys (turned to their positions) and values rounded to
           8 bits and written behind each sequence's tokens, with the scales of
           the blocks they fall into
  attend   attention of each sequence's drafted tokens over such a cache
  verify   which drafted tokens the target's probabilities accept, by given
           random numbers, and the token that follows them
  accept   the accepted tokens of a tree moved up behind the cache's tokens
  pages    the page table of the next step: sequences forked, continued or
           dropped, new pages, partly filled pages copied; or the pool compacted

`own` chooses between the plain form (elementary torch operations) and the
package's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1, "e4m3": 1}
MOST = {"i8": 127.0, "e4m3": 448.0}          # the largest magnitude an element stands for


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # One new token of one sequence: the smallest call, all latency.
        dict(name="append8_one", op="append", B=1, T=1, S=2048, Hq=64, H=8, D=128, q="bf16", kv="e4m3", block=32, layout="shd", rot=128),
        # A decoded cache of two prompts, turned already, into 8-bit pages.
        dict(name="append8_prompt", op="append", B=2, T=8192, S=8192, Hq=0, H=8, D=128, q="bf16", kv="i8", block=16, layout="paged64", rot=0),
        # One token over a short cache of one layer: latency.
        dict(name="attend8_one", op="attend", B=1, T=1, S=2048, Hq=64, H=8, D=128, q="bf16", kv="i8", block=32, layout="shd",
             tree=False, ragged=False),
        # A serving batch: one token each of 32 sequences of very different lengths, in pages.
        dict(name="attend8_batch", op="attend", B=32, T=1, S=16384, Hq=32, H=8, D=128, q="bf16", kv="e4m3", block=16, layout="paged64",
             tree=False, ragged=True),
        # A chain of four drafted tokens over long caches.
        dict(name="attend8_long", op="attend", B=2, T=4, S=131072, Hq=64, H=8, D=128, q="bf16", kv="i8", block=64, layout="hsd",
             tree=False, ragged=False),
        # Trees of 64 drafted tokens for each of 8 sequences: many rows over the same keys.
        dict(name="attend8_tree", op="attend", B=8, T=64, S=8205, Hq=64, H=8, D=128, q="f16", kv="e4m3", block=16, layout="shd",
             tree=True, ragged=True),
        # A chain of four drafted tokens of one sequence.
        dict(name="verify_one", op="verify", B=1, T=5, V=32000, p="f32", draft=True, wide=1, ragged=False),
        # Trees of up to 32 tokens, three to a node, each drawn from the drafting model, of 16 sequences with a large vocabulary.
        dict(name="verify_tree", op="verify", B=16, T=32, V=131072, p="f32", draft=True, wide=3, ragged=True),
        # The accepted tokens of one tree, one layer.
        dict(name="accept_one", op="accept", B=1, T=16, S=4096, H=8, D=128, kv="bf16", layout="shd"),
        # ... of a batch, in pages.
        dict(name="accept_batch", op="accept", B=64, T=64, S=2048, H=8, D=128, kv="bf16", layout="paged16"),
        # Beam search: 32 prompts of up to 8192 tokens with 8 beams each, reordered.
        dict(name="fork_beams", op="fork", B=256, S=8192, H=8, D=128, kv="bf16", page=16, beams=8, room=8, spare=2048),
        # A pool half of whose pages were freed.
        dict(name="compact_pool", op="compact", B=64, S=8192, H=8, D=128, kv="bf16", page=32, gone=0.5, spare=100),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """A case of the listed ones' ranges; sizes over their logarithm, odd ones among them."""
    op = rng.choice(["append", "attend", "attend", "verify", "verify", "accept", "fork", "compact"])
    if op == "verify":
        B, T = _log(rng, 1, 64), _log(rng, 1, 48)
        V = _log(rng, 100, min(200000, 16 * 32 * 131072 // (B * T)))
        return dict(op=op, B=B, T=T, V=V, p=rng.choice(["f32", "f32", "bf16", "f16"]), draft=rng.random() < 0.6, wide=rng.choice([1, 1, 2, 4]),
                    ragged=rng.random() < 0.5)
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    H = rng.choice([1, 2, 4, 5, 8, 8])
    if op in ("fork", "compact"):
        page = rng.choice([16, 16, 32, 64])
        beams = rng.choice([1, 2, 4, 8])
        B = beams * _log(rng, 1, 32)
        S = _log(rng, page, min(8192, 32 * 8192 * 8 * 128 * beams // (B * H * D)))
        c = dict(op=op, B=B, S=S, H=H, D=D, kv=rng.choice(["bf16", "f16"]), page=page, spare=_log(rng, 1, 4000))
        return dict(c, beams=beams, room=_log(rng, 1, 64)) if op == "fork" else dict(c, gone=rng.choice([0.1, 0.5, 0.9]))
    B = _log(rng, 1, 32)
    layout = rng.choice(["shd", "hsd", "paged16", "paged64", "paged256"])
    if op == "accept":
        T = _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, 64), T=T, S=T + _log(rng, 1, 2048), H=H, D=D, kv=rng.choice(["bf16", "f16"]), layout=layout)
    Hq = H * rng.choice([1, 2, 4, 7, 8])
    kv = rng.choice(["i8", "e4m3"])
    q = rng.choice(["bf16", "bf16", "f16"])
    block = rng.choice([16, 16, 32, 64, 128])
    if layout.startswith("paged"):
        block = min(block, int(layout[5:]))
    if op == "append":
        T = _log(rng, 1, min(8192, 2 * 8192 * 8 * 128 // (B * (Hq + H) * D)))
        rot = 0 if kv == "i8" else rng.choice([0, D, D // 2, 20])
        return dict(op=op, B=B, T=T, S=T + _log(rng, 1, 2048), Hq=Hq if rot else 0, H=H, D=D, q=q, kv=kv, block=block, layout=layout, rot=rot)
    T = _log(rng, 1, 128) if rng.random() < 0.6 else 1
    most = min(131072, 2 * 131072 * 8 * 128 // (B * H * D), 8 * 64 * 64 * 8192 * 128 // (B * T * Hq * D))
    return dict(op=op, B=B, T=T, S=T + _log(rng, 1, max(1, most - T)), Hq=Hq, H=H, D=D, q=q, kv=kv, block=block, layout=layout,
                tree=rng.random() < 0.5, ragged=rng.random() < 0.5)


def _lengths(c):
    """(cached tokens, drafted tokens) of each sequence; the case alone decides them."""
    rng = random.Random("%s %d %d %d" % (c["op"], c["B"], c.get("S", 0), c.get("T", 0)))
    T = c.get("T", 0)
    length, drafted = [], []
    for b in range(c["B"]):
        whole = b == 0 or not c.get("ragged")
        length.append(c.get("S", 0) - T if whole else rng.randint(0, c["S"] - T) if "S" in c else 0)
        drafted.append(T if whole else 0 if rng.random() < 0.05 else rng.randint(max(min(1, T), T - 3), T))
    if c["op"] in ("append", "accept"):
        length = [rng.randint(0, c["S"] - T) for _ in length]
    return length, drafted


def _beams(c):
    """(length, parent) of the sequences before a fork; the case alone decides them. Beams of a prompt share its pages."""
    rng = random.Random("%d %d %d" % (c["B"], c["S"], c["beams"]))
    length, parent = [], []
    for first in range(0, c["B"], c["beams"]):
        length += [rng.randint(max(1, c["S"] // 16), c["S"])] * c["beams"]
        ended = rng.random() < 0.1
        parent += [-1 if ended else first + rng.randrange(c["beams"]) for _ in range(c["beams"])]
    return length, parent


# ----------------------------------------------------------------- inputs --
def _page(c):
    return int(c["layout"][5:]) if c["layout"].startswith("paged") else 0


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = random.Random(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def int32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = {"case": c}
    if c["op"] == "verify":
        return _prepare_verify(c, s, g, host, int32)
    B, H, D = c["B"], c["H"], c["D"]
    if c["op"] in ("fork", "compact"):
        return _prepare_pages(c, s, g, normal, int32)

    S, T = c["S"], c["T"]
    length, drafted = _lengths(c)
    s["length"] = int32(length)
    kv = DTYPES[c["kv"]]
    page = _page(c)
    per = -(-S // page) if page else 0

    def cache(mean):
        """Values as a cache holds them, a scale per channel and for keys a mean; in 8 bits with a scale for each block and head."""
        channel = torch.exp(0.8 * normal(H, D)) * 0.7
        bias = mean * normal(H, D)
        first, second = (B * per + 3, page) if page else (B, S)
        hsd = c["layout"] == "hsd"
        t = torch.empty(first, H, second, D, device=dev, dtype=kv).transpose(1, 2) if hsd else torch.empty(first, second, H, D, device=dev, dtype=kv)
        scale = torch.empty(first, -(-second // c["block"]), H, device=dev) if "block" in c else None
        step = max(1, (1 << 25) // (second * H * D))
        for a in range(0, first, step):
            n = min(step, first - a)
            x = (normal(n, second, H, D) + bias) * channel
            if scale is not None:
                short = scale.shape[1] * c["block"] - second
                y = torch.cat((x, x.new_zeros(n, short, H, D)), 1) if short else x
                most = y.view(n, -1, c["block"], H, D).abs().amax((2, 4))
                scale[a:a + n] = most / MOST[c["kv"]] * 1.0001
                x = x / scale[a:a + n].repeat_interleave(c["block"], 1)[:, :second, :, None]
                x = torch.round(x) if kv == torch.int8 else x
            t[a:a + n].copy_(x)
        return t, scale

    s["k"], s["k_scale"] = cache(0.5)
    s["v"], s["v_scale"] = cache(0.0)
    s["table"] = None
    if page:
        order = torch.randperm(B * per + 3, generator=g, device=dev).to(torch.int32)
        s["table"] = order[:B * per].view(B, per).contiguous()
    if c["op"] == "accept":
        s["new_k"], s["new_v"] = normal(B, T, H, D).to(kv), normal(B, T, H, D).to(kv)
        path, count = [], []
        for b in range(B):                   # a way down the tree, from its root
            way = [0]
            while way[-1] + 1 < T and host.random() < 0.8:
                way.append(host.randint(way[-1] + 1, min(T - 1, way[-1] + 9)))
            path.append(way + [-1] * (T - len(way)))
            count.append(len(way))
        s["path"], s["count"] = int32(path), int32(count)
        return s
    s["drafted"] = int32(drafted)
    s["q"] = normal(B, T, c["Hq"], D).to(DTYPES[c["q"]]) if c["Hq"] else None
    if c["op"] == "append":
        spread = torch.exp(0.6 * normal(B, T, 1, 1))          # some tokens are far larger than others
        s["new_k"] = (normal(B, T, H, D) * spread).to(DTYPES[c["q"]])
        s["new_v"] = (normal(B, T, H, D) * spread).to(DTYPES[c["q"]])
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
        s["freq"] = 10000.0 ** (-2.0 * i / c["rot"]) / (2.0 * math.pi) if c["rot"] else None
        return s
    s["tree"] = None
    if c["tree"]:
        trees = []
        for b in range(B):                   # each token's parent is an earlier one, or the cache's last
            seen = [0] * T
            for j in range(T):
                p = host.randint(max(-1, j - 9), j - 1)
                seen[j] = (seen[p] if p >= 0 else 0) | (1 << j)
            trees.append([[bool(m >> j & 1) for j in range(T)] for m in seen])
        s["tree"] = torch.tensor(trees, device=dev)
    return s


def _prepare_verify(c, s, g, host, int32):
    """A target's probabilities, a drafting model's that are near them, and tokens drawn from the drafting model's."""
    B, T, V = c["B"], c["T"], c["V"]
    dev = g.device
    p = torch.empty(B, T, V, device=dev, dtype=DTYPES[c["p"]])
    q = torch.empty_like(p)
    parent = []
    for b in range(B):
        up = [-1] + [max(0, (i - 1) // c["wide"] if c["wide"] > 1 else i - 1) for i in range(1, T)]
        if c["wide"] > 1:                    # some nodes have fewer children
            for i in range(2, T):
                low = max(up[i - 1], i - 2 * c["wide"])
                up[i] = host.randint(low, max(low, min(i - 1, up[i - 1] + 2)))
        parent.append(up)
    s["parent"] = int32(parent) if c["wide"] > 1 else None
    tokens = torch.zeros(B, T, dtype=torch.int32, device=dev)
    for b in range(B):
        logits = 3.0 * torch.randn(T, V, generator=g, device=dev)
        logits[:, :max(1, V // 1000)] += 4.0
        p[b] = torch.softmax(logits, -1)
        logits += 0.7 * torch.randn(T, V, generator=g, device=dev)
        q[b] = torch.softmax(logits, -1)
        if T > 1:
            up = torch.tensor(parent[b][1:], device=dev)
            if c["draft"]:
                tokens[b, 1:] = torch.multinomial(q[b].float()[up], 1, generator=g)[:, 0].int()
            else:                            # the drafting model's most likely ones
                nth = torch.tensor([sum(x == parent[b][i] for x in parent[b][:i]) for i in range(1, T)], device=dev).clamp(max=V - 1)
                best = torch.topk(q[b].float(), min(V, int(nth.max()) + 1), -1).indices
                tokens[b, 1:] = best[up, nth].int()
    s["target"], s["draft"], s["tokens"] = p, q if c["draft"] else None, tokens
    s["drafted"] = int32(_lengths(c)[1])
    s["uniform"] = torch.rand(B, T, generator=g, device=dev)
    return s


def _prepare_pages(c, s, g, normal, int32):
    """Tables whose sequences share the pages of their prompts, or that have lost some of their sequences."""
    B, S, page = c["B"], c["S"], c["page"]
    dev = g.device
    per = -(-S // page)
    if c["op"] == "fork":
        length, parent = _beams(c)
        need = sum(-(-length[b] // page) for b in range(0, B, c["beams"])) + B
        pages = need + B * (c["room"] // page + 2) + c["spare"]
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).tolist()
        table, at = [], 0
        for first in range(0, B, c["beams"]):
            n = -(-length[first] // page)
            shared = order[at:at + n - 1]
            at += n - 1
            for _ in range(c["beams"]):      # all but the last page are the prompt's
                table.append(shared + [order[at]] + [-1] * (per + c["room"] // page + 1 - n))
                at += 1
        s["parent"] = int32(parent)
    else:
        length = _kept(c)
        pages = B * per + c["spare"]
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[:B * per].view(B, per).tolist()
        table = [order[b][:-(-length[b] // page)] + [-1] * (per - -(-length[b] // page)) for b in range(B)]
    s["table"], s["length"], s["pages"] = int32(table), int32(length), pages
    s["k"], s["v"] = (torch.empty(pages, page, c["H"], c["D"], device=dev, dtype=DTYPES[c["kv"]]) for _ in "kv")
    for t in (s["k"], s["v"]):
        for part in t.chunk(max(1, t.numel() >> 27), 0):
            part.copy_(normal(*part.shape))
    return s


def _kept(c):
    """Lengths of the sequences before a compaction; those that ended have none. The case alone decides them."""
    rng = random.Random("%d %d" % (c["B"], c["S"]))
    return [0 if rng.random() < c["gone"] else rng.randint(max(1, c["S"] // 4), c["S"]) for _ in range(c["B"])]


# ------------------------------------------------------------ plain forms --
def _bits(t):
    """A view that every indexing operation knows: FP8 values as bytes."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _rows(cache, table, at, unit=1):
    """Index of the first two dims of a cache (or of its scales, one for each `unit` tokens) for tokens at [sequences, ...]."""
    b = torch.arange(at.shape[0], device=at.device).view(-1, *[1] * (at.dim() - 1))
    if table is None:
        return b.expand_as(at), at // unit
    page = cache.shape[1] * unit
    return table.long()[b, at // page], at % page // unit


def _append(s):
    c = s["case"]
    B, T, S, H, D, unit = c["B"], c["T"], c["S"], c["H"], c["D"], c["block"]
    dev = s["new_k"].device
    length = s["length"].long()

    def turned(x):
        x = x.float()
        if not c["rot"]:
            return x
        half = c["rot"] // 2
        turns = (length[:, None] + torch.arange(T, device=dev)).double()[..., None] * s["freq"]
        angle = (turns - torch.round(turns)) * (2.0 * math.pi)
        cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]), -1)

    # a window of whole blocks that holds the new tokens; t: which of them is at a place
    blocks = -(-T // unit) + 1
    at = (length // unit * unit)[:, None] + torch.arange(blocks * unit, device=dev)
    t = at - length[:, None]
    new = (t >= 0) & (t < s["drafted"][:, None]) & (at < S)
    place = at.clamp(max=S - 1)
    most = MOST[c["kv"]]

    def written(cache, scale, x):
        x = torch.where(new[..., None, None], x.gather(1, t.clamp(0, T - 1)[..., None, None].expand(-1, -1, H, D)), 0.0)
        x = x.view(B, blocks, unit, H, D)
        top = x.abs().amax((2, 4))                                        # [B, blocks, H]
        part, power = torch.frexp(top)                                    # the smallest power of two that holds it
        down = 7 if most == 127.0 else 9
        power = torch.where(part * 2.0 ** down <= most, power - down, power - down + 1).clamp(min=-60)
        need = torch.ldexp(torch.ones_like(top), power)
        rows = _rows(scale, s["table"], place.view(B, blocks, unit)[:, :, 0], unit)
        before = scale[rows]
        earlier = (t.view(B, blocks, unit)[:, :, 0] < 0)[..., None]
        now = torch.where(earlier & (top <= before * most), before, need)
        old = _bits(cache)[_rows(cache, s["table"], place)].view(cache.dtype).float().view(B, blocks, unit, H, D)
        ratio = torch.where(earlier & (before != now), before / now, 1.0)[:, :, None, :, None]
        y = torch.where(new.view(B, blocks, unit)[..., None, None], x / now[:, :, None, :, None], old * ratio)
        y = (torch.round(y) if most == 127.0 else y).clamp(-most, most).to(cache.dtype).view(B, blocks * unit, H, D)
        touched = new.view(B, blocks, unit).any(-1)
        put = (new | ((t < 0) & touched.repeat_interleave(unit, 1)))
        _bits(cache)[tuple(r[put] for r in _rows(cache, s["table"], place))] = _bits(y)[put]
        scale[tuple(r[touched] for r in rows)] = now[touched]

    written(s["k"], s["k_scale"], turned(s["new_k"]))
    written(s["v"], s["v_scale"], s["new_v"].float())
    got = {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return dict(got, q=turned(s["q"]).to(s["q"].dtype)) if c["Hq"] else got


def _attend(s):
    c = s["case"]
    B, T, S, H, D = c["B"], c["T"], c["S"], c["H"], c["D"]
    G = c["Hq"] // H
    dev = s["q"].device

    def whole(cache, scale):         # [B, H, S, D] in 32 bits
        if s["table"] is not None:
            cache = _bits(cache)[s["table"].long()].flatten(1, 2)[:, :S].view(cache.dtype)
            scale = scale[s["table"].long()].flatten(1, 2)
        return cache.permute(0, 2, 1, 3).float() * scale.repeat_interleave(c["block"], 1)[:, :S].transpose(1, 2)[..., None]

    at = torch.arange(S, device=dev)[None, None, :]
    j = at - s["length"][:, None, None]                                   # which drafted token, by cache slot
    i = torch.arange(T, device=dev)[None, :, None]
    if s["tree"] is None:
        seen = j <= i
    else:
        seen = (j < 0) | (torch.gather(s["tree"], 2, j.clamp(0, T - 1).expand(B, T, S)) & (j < T))
    seen = seen & (i < s["drafted"][:, None, None]) & (j < s["drafted"][:, None, None])
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    w = torch.matmul(whole(s["k"], s["k_scale"]), q.transpose(-1, -2).contiguous()).transpose(-1, -2)
    w = w.mul_(1.0 / math.sqrt(D)).view(B, H, T, G, S).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    w = w.div_(torch.where(total == 0, torch.ones_like(total), total))
    out = torch.matmul(w.view(B, H, T * G, S), whole(s["v"], s["v_scale"])).view(B, H, T, G, D)
    lse = (total.log() + top)[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, T, c["Hq"], D).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, T, c["Hq"])}


def _verify(s):
    """The drafted tokens in their order: each is tried if its parent is where its sequence's way has come to.

    With c the multiple of the drafting model's probabilities q that rejected
    siblings took from the target's p, what is left is max(p - c q, 0), of sum
    `mass`; without q a rejected token itself is taken out.
    """
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    p, q, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniform"].double()
    dev = p.device
    row, node = torch.arange(B, device=dev), torch.arange(T, device=dev)
    parent = s["parent"].long() if s["parent"] is not None else (node - 1).expand(B, T)
    there = node < s["drafted"][:, None]
    siblings = (parent[:, :, None] == parent[:, None, :]) & (node[:, None] > node)
    again = (siblings & (tokens[:, :, None] == tokens[:, None, :])).any(-1) & (q is None)
    at = torch.zeros(B, dtype=torch.long, device=dev)
    path = torch.full((B, T), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.long, device=dev)
    going = s["drafted"] > 0
    much = torch.zeros(B, dtype=torch.float64, device=dev)
    mass = torch.ones_like(much)
    for i in range(1, T):
        mine = going & there[:, i] & (parent[:, i] == at)
        x = tokens[:, i]
        qx = q[row, at, x].double() if q is not None else torch.ones_like(mass)
        px = p[row, at, x].double()
        left = (px - much * qx).clamp(min=0.0) if q is not None else px
        yes = mine & (left > 0) & ~again[:, i] & (u[:, i] * qx * mass < left)
        no = mine & ~yes
        much = torch.where(yes, 0.0, torch.where(no, much + mass, much))
        if q is None:
            less = torch.where(again[:, i], mass, mass - px)
        elif s["parent"] is None:    # nothing more is tried there
            less = mass
        else:
            less = (p[row, at].double() - much[:, None] * q[row, at].double()).clamp_(min=0.0).sum(-1)
        mass = torch.where(yes, 1.0, torch.where(no, less, mass))
        at = torch.where(yes, i, at)
        path = torch.where(yes[:, None] & (node == count[:, None]), i, path)
        count = count + yes
    left = p[row, at].double()
    if q is not None:
        left = (left - much[:, None] * q[row, at].double()).clamp_(min=0.0)
    else:
        tried = there & (parent == at[:, None]) & (node > 0)
        left = torch.cat((left, left.new_zeros(B, 1)), 1).scatter_(1, torch.where(tried, tokens, V), 0.0)[:, :V]
    none = (left > 0).sum(-1) == 0
    left = torch.where(none[:, None], p[row, at].double(), left)
    sums = left.cumsum(-1)
    token = (sums <= u[:, :1] * sums[:, -1:]).sum(-1)
    last = (left > 0).to(torch.int32).mul(torch.arange(1, V + 1, device=dev)).amax(-1) - 1
    token = torch.minimum(token, last)
    return {"path": torch.where(going[:, None], path, -1), "count": torch.where(going, count, 0).int(),
            "token": torch.where(going, token, -1).int()}


def _accept(s):
    c = s["case"]
    j = torch.arange(c["T"], device=s["path"].device)
    at = s["length"].long()[:, None] + j
    for cache, new in ((s["k"], s["new_k"]), (s["v"], s["new_v"])):       # the drafted tokens, as they were appended
        cache[_rows(cache, s["table"], at)] = new
    src = torch.where(j < s["count"][:, None], s["path"].long(), j) + s["length"].long()[:, None]
    for cache in (s["k"], s["v"]):
        cache[_rows(cache, s["table"], at)] = cache[_rows(cache, s["table"], src)]
    return {"k": s["k"], "v": s["v"]}


def _fork(s):
    c = s["case"]
    table, page, pages = s["table"].long(), c["page"], s["pages"]
    B, E = s["parent"].shape[0], table.shape[1]
    dev = table.device
    live = (s["parent"] >= 0) & (s["parent"] < table.shape[0])
    src = torch.where(live, s["parent"], 0).long()
    n = torch.where(live, s["length"].long()[src].clamp(0, E * page), 0)
    rows, e = table[src], torch.arange(E, device=dev)
    there = (rows >= 0) & (rows < pages)
    full, part = n // page, n % page > 0
    kept = (e < full[:, None]) & there
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used[torch.where(kept, rows, pages)] = True
    # a partly filled last page stays with the first sequence that has it
    last = rows.gather(1, full.clamp(max=E - 1)[:, None])[:, 0]
    has = part & (last >= 0) & (last < pages)
    b = torch.arange(B, device=dev)
    first = torch.full((pages + 1,), B, device=dev).scatter_reduce_(0, torch.where(has, last, pages), b, "amin")
    at = torch.where(has, last, pages)
    mine = has & ~used[at] & (first[at] == b)
    copy = has & ~mine
    used[torch.where(mine, last, pages)] = True
    free = ~used[:pages]
    order = torch.full((pages + 1,), -1, device=dev).scatter_(0, torch.where(free, free.long().cumsum(0) - 1, pages), torch.arange(pages, device=dev))
    order[pages] = -1                # of pages in use, which all went there
    end = ((n + c["room"] + page - 1) // page).clamp(max=E)
    fresh = live[:, None] & (e >= (full + (part & ~copy).long())[:, None]) & (e < end[:, None])
    given = order[(fresh.flatten().long().cumsum(0) - 1).clamp(0, pages)].view(B, E)
    new = torch.where(kept, rows, -1)
    new = torch.where(mine[:, None] & (e == full[:, None]), rows, new)
    new = torch.where(fresh, given, new)
    to = new.gather(1, full.clamp(max=E - 1)[:, None])[:, 0]
    copy = copy & (to >= 0)
    moves = torch.stack((torch.where(copy, last, -1), torch.where(copy, to, -1)), 1)
    for pool in (s["k"], s["v"]):
        pool[to[copy]] = pool[last[copy]]
    return {"table": new.int(), "length": n.int(), "moves": moves.int(), "left": (free.sum() - fresh.sum()).int().view(1), "k": s["k"], "v": s["v"]}


def _compact(s):
    c = s["case"]
    table, page, pages = s["table"].long(), c["page"], s["pages"]
    B, E = table.shape
    dev = table.device
    n = s["length"].long().clamp(0, E * page)
    kept = (torch.arange(E, device=dev) < ((n + page - 1) // page)[:, None]) & (table >= 0) & (table < pages)
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used[torch.where(kept, table, pages)] = True
    used = used[:pages]
    count = used.sum()
    at = torch.arange(pages, device=dev)
    src, dst = (used & (at >= count)).nonzero()[:, 0], (~used & (at < count)).nonzero()[:, 0]
    to = at.clone()
    to[src] = dst
    moves = torch.full((min(B * E, pages // 2), 2), -1, dtype=torch.int32, device=dev)
    moves[:src.numel(), 0], moves[:src.numel(), 1] = src.int(), dst.int()
    for pool in (s["k"], s["v"]):
        pool[dst] = pool[src]
    return {"table": torch.where(kept, to[torch.where(kept, table, 0)], -1).int(), "moves": moves, "used": count.int().view(1), "k": s["k"], "v": s["v"]}


def run(s):
    c = s["case"]
    if not own:
        return {"append": _append, "attend": _attend, "verify": _verify, "accept": _accept, "fork": _fork, "compact": _compact}[c["op"]](s)
    from lossless_bf16_tensor_amd import kv
    if c["op"] == "append":
        q = kv.append(s["q"], s["new_k"], s["new_v"], s["k"], s["v"], s["length"], s["freq"], table=s["table"], drafted=s["drafted"],
                      k_scale=s["k_scale"], v_scale=s["v_scale"])
        got = {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        return dict(got, q=q) if c["Hq"] else got
    if c["op"] == "attend":
        lse = torch.empty(c["B"], c["T"], c["Hq"], device=s["q"].device)
        out = kv.attend(s["q"], s["k"], s["v"], s["length"], table=s["table"], tree=s["tree"], drafted=s["drafted"], lse=lse,
                        k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if c["op"] == "verify":
        path, count, token = kv.verify(s["tokens"], s["target"], s["uniform"], draft=s["draft"], parent=s["parent"], drafted=s["drafted"])
        return {"path": path, "count": count, "token": token}
    if c["op"] == "accept":
        kv.append(None, s["new_k"], s["new_v"], s["k"], s["v"], s["length"], table=s["table"])
        kv.accept(s["k"], s["v"], s["length"], s["path"], s["count"], table=s["table"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "fork":
        table, length, moves, left = kv.fork(s["table"], s["length"], s["parent"], s["pages"], c["page"], room=c["room"])
        kv.copy_pages(moves, s["k"], s["v"])
        return {"table": table, "length": length, "moves": moves, "left": left, "k": s["k"], "v": s["v"]}
    table, moves, used = kv.compact(s["table"], s["length"], s["pages"], c["page"])
    kv.copy_pages(moves, s["k"], s["v"])
    return {"table": table, "moves": moves, "used": used, "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------- work --
def work(c):
    """Each input read once and each output written once."""
    B = c["B"]
    if c["op"] == "verify":          # the row that the next token is drawn from, and of the drafting model's the same one
        return {"bytes": B * c["V"] * SIZE[c["p"]] * (2 if c["draft"] else 1) + 20 * B * c["T"], "flops": 3 * B * c["V"]}
    H, D = c["H"], c["D"]
    es = SIZE[c["kv"]]
    if c["op"] == "fork":
        length, parent = _beams(c)
        n = [length[p] if p >= 0 else 0 for p in parent]
        shared = len({p for p in parent if p >= 0 and length[p] % c["page"]})
        copies = sum(p >= 0 and length[p] % c["page"] > 0 for p in parent) - shared
        return {"bytes": 8 * sum(-(-x // c["page"]) for x in n) + 4 * copies * c["page"] * H * D * es, "flops": 0}
    if c["op"] == "compact":
        used = sum(-(-x // c["page"]) for x in _kept(c))
        pages = B * -(-c["S"] // c["page"]) + c["spare"]
        return {"bytes": 8 * used + 4 * (used * (pages - used) // pages) * c["page"] * H * D * es, "flops": 0}
    length, drafted = _lengths(c)
    n = B * c["T"] * H * D
    if c["op"] == "accept":          # the append before it, and about five tokens of a way moved
        return {"bytes": 4 * n * es + 4 * min(5, c["T"]) * B * H * D * es, "flops": 0}
    if c["op"] == "append":
        nq = B * c["T"] * c["Hq"] * D
        return {"bytes": 2 * nq * 2 + 2 * n * (2 + es) + 8 * n // (D * c["block"]), "flops": 6 * (nq + n) * c["rot"] // (2 * D) + 6 * n}
    seen = [m + t if t else 0 for m, t in zip(length, drafted)]
    rows = B * c["T"] * c["Hq"]
    return {"bytes": 2 * sum(seen) * H * (D * es + 4 / c["block"]) + 2 * rows * D * 2 + 4 * rows,
            "flops": 4 * D * c["Hq"] * sum(m * t for m, t in zip(seen, drafted))}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The definitions in 64 bits, one sequence and head at a time. Whole numbers (verify, tables) have no error to tell."""
    if case["op"] == "verify":
        return None
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64
    if c["op"] in ("fork", "compact"):
        return _exact_pages(c, s)
    length, T, H, D = s["length"].tolist(), c["T"], c["H"], c["D"]

    def slots(b, n0, n1, unit=1):    # (first, second) indexes of tokens [n0, n1) of sequence b, or of their scales
        n = torch.arange(n0, n1, device=s["k"].device)
        if s["table"] is None:
            return torch.full_like(n, b), n // unit
        page = s["k"].shape[1]
        return s["table"][b].long()[n // page], n % page // unit

    if c["op"] == "accept":
        k, v = s["k"].to(f64), s["v"].to(f64)
        for b, n in enumerate(length):
            for whole, new in ((k, s["new_k"]), (v, s["new_v"])):
                rows = new[b].to(f64)
                for j, i in enumerate(s["path"][b, :int(s["count"][b])].tolist()):
                    rows[j] = new[b, i].to(f64)
                whole[slots(b, n, n + T)] = rows
        return {"k": k, "v": v}
    if c["op"] == "append":
        got = {"k": s["k"].to(f64), "v": s["v"].to(f64), "k_scale": s["k_scale"].to(f64), "v_scale": s["v_scale"].to(f64)}
        most, unit = MOST[c["kv"]], c["block"]

        def turned(x, n):
            x = x.to(f64)
            half = c["rot"] // 2
            if not half:
                return x
            turn = torch.outer(torch.arange(n, n + T, device=x.device, dtype=f64), s["freq"])
            z = torch.polar(torch.ones_like(turn), torch.remainder(turn, 1.0) * 2.0 * math.pi)[:, None]
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * z
            return torch.cat((z.real, z.imag, x[..., 2 * half:]), -1)

        for b, n in enumerate(length):
            t = int(s["drafted"][b])
            for name, x in (("k", turned(s["new_k"][b], n)), ("v", s["new_v"][b].to(f64))):
                for n0 in range(n // unit * unit, n + t, unit):
                    lo, hi = max(n, n0), min(n + t, n0 + unit)
                    top = x[lo - n:hi - n].abs().amax((0, 2))
                    at = tuple(i[0] for i in slots(b, n0, n0 + 1, unit))
                    old = got[name + "_scale"][at].clone()
                    fits = torch.exp2(torch.ceil(torch.log2(top / most)).clamp(min=-60.0))
                    now = torch.where(top <= old * most, old, fits) if n0 < n else fits
                    got[name + "_scale"][at] = now
                    y = x[lo - n:hi - n]
                    if n0 < n:
                        y = torch.cat((got[name][slots(b, n0, n)] * old[:, None], y))
                    y = y / now[:, None]
                    # to the nearest step of the element's type, ties to even
                    step = torch.ones_like(y) if most == 127.0 else torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
                    got[name][slots(b, n0 if n0 < n else lo, hi)] = torch.round(y / step) * step
        if c["Hq"]:
            got["q"] = torch.stack([turned(s["q"][b], n) for b, n in enumerate(length)])
        return got

    G = c["Hq"] // H
    out = torch.zeros(c["B"], T, c["Hq"], D, dtype=f64, device=s["q"].device)
    lse = torch.full((c["B"], T, c["Hq"]), -math.inf, dtype=f64, device=out.device)
    for b, (n, t) in enumerate(zip(length, s["drafted"].tolist())):
        if not t:
            continue
        k, v = (_bits(s[x])[slots(b, 0, n + t)].view(s[x].dtype) for x in "kv")
        ks, vs = (s[x][slots(b, 0, n + t, c["block"])].to(f64) for x in ("k_scale", "v_scale"))
        hidden = torch.ones(t, t, device=out.device).triu(1).bool() if s["tree"] is None else ~s["tree"][b, :t, :t]
        for h in range(H):
            kk, vv = k[:, h].to(f64) * ks[:, h, None], v[:, h].to(f64) * vs[:, h, None]
            for a in range(h * G, h * G + G):
                w = s["q"][b, :t, a].to(f64) @ kk.t() / math.sqrt(D)
                w[:, n:] = w[:, n:].masked_fill(hidden, -math.inf)
                lse[b, :t, a] = torch.logsumexp(w, -1)
                p = torch.exp(w - torch.where(torch.isinf(lse[b, :t, a]), 0.0, lse[b, :t, a])[:, None])
                out[b, :t, a] = p @ vv
    return {"out": out, "lse": lse}


def _exact_pages(c, s):
    """Pages handed out one at a time; only the pools' values have an error to tell."""
    if s["k"].numel() > 1 << 28:
        return None
    table, length, page, pages = s["table"].tolist(), s["length"].tolist(), c["page"], s["pages"]
    moves = []
    if c["op"] == "fork":
        parent = s["parent"].tolist()
        seqs = [(table[p], length[p]) if 0 <= p < len(table) else ([], 0) for p in parent]
        taken = {x for row, n in seqs for x in row[:n // page]}
        lasts = set()
        want = []                    # what each sequence needs, in order: a copy of its last page, or empty pages
        for row, n in seqs:
            if not n:
                want.append([])
                continue
            end = min(-(-(n + c["room"]) // page), len(row))
            mine = n % page > 0 and row[n // page] not in taken | lasts
            if mine:
                lasts.add(row[n // page])
            copied = n % page > 0 and not mine
            want.append([row[n // page] if copied and i == 0 else -1 for i in range(end - n // page - (1 if mine else 0))])
        free = (x for x in range(pages) if x not in taken | lasts)
        for pieces in want:
            for src in pieces:
                dst = next(free)
                moves += [(src, dst)] if src >= 0 else []
    else:
        used = sorted({x for row, n in zip(table, length) for x in row[:-(-n // page)]})
        holes = sorted(set(range(len(used))) - set(used))
        moves = list(zip([x for x in used if x >= len(used)], holes))
    got = {"k": s["k"].double(), "v": s["v"].double()}
    for x in "kv":
        for src, dst in moves:
            got[x][dst] = s[x][src].double()
    return dict(got, **({"table": None, "length": None, "moves": None, "left": None} if c["op"] == "fork" else {"table": None, "moves": None, "used": None}))
