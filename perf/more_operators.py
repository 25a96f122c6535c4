"""Measured cases of the paged cache's operators for long contexts and drafted
tokens: what each computes, in plain torch and through the library, and what
it cannot do without.

``window``  causal attention over the cache with a sliding window and a few
            first tokens that stay visible, prompts and single tokens
``tree``    attention of a tree of drafted tokens over the cache
``append``  one step's keys (rotated) and values written to an 8-bit cache and
            read back
``read``    tokens of an 8-bit cache read back as 16- or 32-bit values
``verify``  a verification step's bookkeeping: rows grow by their drafted
            tokens, the accepted ones move together and the rest is dropped

A pool of pages is a tensor [pages, rows, heads, dim] or, where a case says
``heads_first``, [pages, heads, rows, dim].  In a 16-bit pool `rows` is the
slots of a page.  In an 8-bit one (``fmt`` int8 or e4m3, a byte an element) the
slots are followed by ceil(2 * slots / dim) rows that hold, for each head, the
slots' scales in bf16.  Page tables, lengths and counts are int32.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TOP = {"int8": 127.0, "e4m3": 448.0}


# ---- the cases -------------------------------------------------------------

def listed():
    return [
        # four short chats' next token, a window of 128: the smallest call
        dict(name="window 4 x 1 of 512 f16", op="window", dtype="f16", fmt="same", batch=4, q_len=1, heads=8,
             kv_heads=2, dim=64, slots=16, ctx=512, window=128, sinks=4, ragged=False, heads_first=False),
        # a large batch's next tokens over long contexts, the cache in 8 bits
        dict(name="window 64 x 1 of 32768 e4m3", op="window", dtype="bf16", fmt="e4m3", batch=64, q_len=1, heads=32,
             kv_heads=8, dim=128, slots=16, ctx=32768, window=8192, sinks=4, ragged=False, heads_first=False),
        # the later half of a long prompt
        dict(name="window 8192 of 16384 bf16", op="window", dtype="bf16", fmt="same", batch=1, q_len=8192, heads=32,
             kv_heads=8, dim=128, slots=16, ctx=16384, window=4096, sinks=4, ragged=False, heads_first=False),
        # chunks of several prompts, padded to the longest, odd sizes, the cache in 8 bits
        dict(name="window 5 x 777 of 2000 int8", op="window", dtype="f16", fmt="int8", batch=5, q_len=777, heads=20,
             kv_heads=4, dim=80, slots=48, ctx=2000, window=300, sinks=3, ragged=True, heads_first=True),
        # one chat's drafted tokens, latency counts
        dict(name="tree 2 x 13 of 700 f16", op="tree", dtype="f16", fmt="same", batch=2, q_len=13, heads=8,
             kv_heads=2, dim=64, slots=16, ctx=700, window=0, sinks=0, ragged=True, heads_first=False),
        # a batch's drafted trees over long contexts
        dict(name="tree 16 x 61 of 16384 bf16", op="tree", dtype="bf16", fmt="same", batch=16, q_len=61, heads=32,
             kv_heads=8, dim=128, slots=32, ctx=16384, window=0, sinks=0, ragged=True, heads_first=True),
        # one decode step's tokens
        dict(name="append 64 bf16 e4m3", op="append", dtype="bf16", fmt="e4m3", tokens=64, rows=64, heads=32,
             kv_heads=8, dim=128, rot=128, layout="half", slots=16, row_tokens=4096, heads_first=False),
        # a prompt's chunk, part of each head rotated in pairs
        dict(name="append 8191 f16 int8", op="append", dtype="f16", fmt="int8", tokens=8191, rows=4, heads=32,
             kv_heads=8, dim=128, rot=64, layout="interleaved", slots=48, row_tokens=4096, heads_first=True),
        # a short row taken out of the cache
        dict(name="read 300 f16 int8", op="read", dtype="f16", fmt="int8", tokens=300, kv_heads=4, dim=96, slots=16,
             pages=400, heads_first=False),
        # long contexts taken out for a dense product
        dict(name="read 65536 bf16 e4m3", op="read", dtype="bf16", fmt="e4m3", tokens=65536, kv_heads=8, dim=128,
             slots=16, pages=6000, heads_first=False),
        # one chat's accepted tokens, two layers
        dict(name="verify 2 x 13, 4 pools", op="verify", fmt="same", batch=2, nodes=13, ctx=700, kv_heads=2, dim=64,
             slots=16, pools=4, heads_first=False),
        # a batch's, eight layers in 8 bits
        dict(name="verify 128 x 64, 16 pools 8 bits", op="verify", fmt="int8", batch=128, nodes=64, ctx=2048,
             kv_heads=8, dim=128, slots=16, pools=16, heads_first=False),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["window", "window", "tree", "append", "read", "verify"])
    kv = rng.choice([1, 2, 4, 8])
    first = rng.random() < 0.5
    fmt = rng.choice(["same", "int8", "e4m3"])
    slots = rng.choice([1, 8, 16, 32, 48, 64, 100, 256])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    if op in ("window", "tree"):
        if op == "window":
            q_len = rng.choice([1, 1, _between(rng, 2, 2048)])
            window = rng.choice([0, _between(rng, 1, 4096), _between(rng, 1, 4096)])
        else:
            q_len = _between(rng, 2, 200)
            window = rng.choice([0, 0, _between(rng, 1, 4096)])
        # as many sequences as the work of the largest case and a few GiB of plain scores allow
        ctx = q_len + _between(rng, 1, 16384)
        most = max(1, min(64, (1 << 29) // (4 * kv * q_len * ctx), (1 << 28) // (kv * ctx * dim)))
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), fmt=fmt, batch=_between(rng, 1, most), q_len=q_len,
                    heads=kv * rng.choice([1, 2, 4, 5]), kv_heads=kv, dim=dim, slots=slots, ctx=ctx, window=window,
                    sinks=rng.choice([0, 1, 4, 16]) if window else 0, ragged=rng.random() < 0.5, heads_first=first)
    fmt8 = rng.choice(["int8", "e4m3"])
    if op == "append":
        rows = _between(rng, 1, 64)
        tokens = _between(rng, rows, 4096)
        return dict(op=op, dtype=rng.choice(["f16", "bf16"]), fmt=fmt8, tokens=tokens, rows=rows,
                    heads=kv * rng.randint(1, 4), kv_heads=kv, dim=dim, rot=2 * rng.randint(1, dim // 2),
                    layout=rng.choice(["half", "interleaved"]), slots=slots,
                    row_tokens=-(-tokens // rows) + _between(rng, 1, 512), heads_first=first)
    if op == "read":
        tokens = _between(rng, 1, 16384)
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), fmt=fmt8, tokens=tokens, kv_heads=kv, dim=dim,
                    slots=slots, pages=-(-tokens // slots) + rng.randint(0, 50), heads_first=first)
    return dict(op=op, fmt=rng.choice(["same", "same", "int8"]), batch=_between(rng, 1, 64), nodes=_between(rng, 2, 100),
                ctx=_between(rng, 1, 1000), kv_heads=rng.choice([1, 2, 4]), dim=rng.choice([64, 80, 128]), slots=slots,
                pools=rng.choice([1, 2, 3, 8]), heads_first=first)


# ---- inputs ----------------------------------------------------------------

def _ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).to(DEV)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _rows(c):
    """Rows of dim elements that a head has in a page."""
    return c["slots"] + (0 if c["fmt"] == "same" else -(-2 * c["slots"] // c["dim"]))


def _empty_pool(c, pages, dtype):
    a, b = (c["kv_heads"], _rows(c)) if c["heads_first"] else (_rows(c), c["kv_heads"])
    return torch.zeros((pages, a, b, c["dim"]), device=DEV, dtype=dtype)


def _filled_pool(g, c, pages):
    """A pool of normal values: in 16 bits, or as 8-bit codes with the scales of such values."""
    if c["fmt"] == "same":
        pool = _empty_pool(c, pages, TYPES[c["dtype"]])
        return pool.copy_(torch.randn(pool.shape, generator=g, device=DEV, dtype=torch.float32))
    pool = _empty_pool(c, pages, torch.uint8)
    top = TOP[c["fmt"]]
    for at in range(0, pages, 8192):  # a part of the pool after the other: the values take four times its memory
        part = pool[at:at + 8192]
        heads = _heads(part, c)                                  # [pages, heads, rows, dim]
        x = torch.randn((part.shape[0], c["kv_heads"], c["slots"], c["dim"]), generator=g, device=DEV)
        scale = _scale(x, top)
        x = x / scale.float()
        heads[:, :, :c["slots"]] = x.round().to(torch.int8).view(torch.uint8) if c["fmt"] == "int8" else \
            x.to(torch.float8_e4m3fn).view(torch.uint8)
        tail = torch.zeros((part.shape[0], c["kv_heads"], (_rows(c) - c["slots"]) * c["dim"] // 2), device=DEV,
                           dtype=torch.bfloat16)
        tail[..., :c["slots"]] = scale[..., 0]
        heads[:, :, c["slots"]:] = tail.flatten().view(torch.uint8).view(part.shape[0], c["kv_heads"], -1, c["dim"])
    return pool


def _scale(x, top):
    """The scale of each head: its largest magnitude over the largest code, rounded up to bf16."""
    bits = (x.abs().amax(-1, keepdim=True).double() / top).float().view(torch.int32)
    return ((bits + 0xFFFF) & -0x10000).view(torch.float32).bfloat16()


def _heads(pool, c):
    """A pool as [pages, heads, rows, dim], without a copy."""
    return pool if c["heads_first"] else pool.transpose(1, 2)


def _held(c):
    """Tokens of each sequence: from all of ctx down to half of it, the last of several a row that was just given up."""
    n = c["batch"]
    held = [c["ctx"] - i * (c["ctx"] // 2) // n for i in range(n)]
    if n > 2:
        held[-1] = 0
    return held


def _counts(c):
    """Queries of each sequence, at most its tokens for a tree."""
    n, held = c["q_len"], _held(c)
    some = [n - (i * (n // 2) // c["batch"] if c["ragged"] else 0) for i in range(c["batch"])]
    return [min(a, b) for a, b in zip(some, held)] if c["op"] == "tree" else some


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": case}
    getattr(_Inputs, case["op"])(case, g, rng, s)
    if own:  # the maps, plan and workspace that a program makes once for its buffers
        import async_tensor_tile_amd as att
        s["att"] = att
        getattr(_Handles, case["op"])(att, case, s)
    return s


class _Inputs:
    @staticmethod
    def window(c, g, rng, s):
        shape = (c["batch"], c["q_len"], c["heads"], c["dim"])
        s["q"] = _normal(g, shape, TYPES[c["dtype"]])
        s["o"] = torch.ones_like(s["q"])                         # what a sequence does not ask for stays as it was
        s["lse"] = torch.ones(shape[:3], device=DEV, dtype=torch.float32)
        each = -(-c["ctx"] // c["slots"])
        pages = c["batch"] * each + 3
        s["k_pool"], s["v_pool"] = _filled_pool(g, c, pages), _filled_pool(g, c, pages)
        s["table"] = _ints(rng.permutation(pages)[:c["batch"] * each].reshape(c["batch"], each))
        order = rng.permutation(c["batch"])                      # the sequences' rows in any order
        lens = np.zeros(c["batch"], dtype=np.int32)
        lens[order] = _held(c)
        s["rows"], s["lens"], s["count"] = _ints(order), _ints(lens), _ints(_counts(c))
        s["scale"] = 1.0 / math.sqrt(c["dim"])

    @staticmethod
    def tree(c, g, rng, s):
        _Inputs.window(c, g, rng, s)
        # a drafted tree: each token follows one of the few before it, some follow the context itself
        j = np.arange(c["q_len"])
        parent = j - rng.integers(1, 9, (c["batch"], c["q_len"]))
        s["parent"] = _ints(np.maximum(parent, -1))

    @staticmethod
    def append(c, g, rng, s):
        t, n, r = TYPES[c["dtype"]], c["tokens"], c["rows"]
        s["q"] = _normal(g, (n, c["heads"], c["dim"]), t)
        s["k"] = _normal(g, (n, c["kv_heads"], c["dim"]), t)
        s["v"] = _normal(g, (n, c["kv_heads"], c["dim"]), t)
        s["q_out"], s["k_back"], s["v_back"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
        row_pages = -(-c["row_tokens"] // c["slots"])
        pages = r * row_pages
        s["k_pool"], s["v_pool"] = _empty_pool(c, pages, torch.uint8), _empty_pool(c, pages, torch.uint8)
        s["table"] = _ints(rng.permutation(pages).reshape(r, row_pages))
        per = np.bincount(np.arange(n) % r, minlength=r)         # rows differ by at most one token
        held = [int(rng.integers(0, c["row_tokens"] - p + 1)) for p in per]
        s["rows"] = _ints(np.repeat(np.arange(r), per))
        s["at"] = _ints(np.concatenate([h + np.arange(p) for h, p in zip(held, per)]))
        s["pos"] = s["at"] + int(rng.integers(0, 1 << 16))       # behind a prefix of that length
        s["freq"] = torch.from_numpy(_frequencies(c)).to(DEV)

    @staticmethod
    def read(c, g, rng, s):
        s["k_pool"], s["v_pool"] = _filled_pool(g, c, c["pages"]), _filled_pool(g, c, c["pages"])
        s["table"] = _ints(rng.permutation(c["pages"])[None])
        start = int(rng.integers(0, c["pages"] * c["slots"] - c["tokens"] + 1))
        s["at"] = _ints(start + np.arange(c["tokens"]))
        s["rows"] = torch.zeros_like(s["at"])
        shape = (c["tokens"], c["kv_heads"], c["dim"])
        s["k"], s["v"] = (torch.empty(shape, device=DEV, dtype=TYPES[c["dtype"]]) for _ in "kv")

    @staticmethod
    def verify(c, g, rng, s):
        n, w, slots = c["batch"], c["nodes"], c["slots"]
        base = rng.integers((c["ctx"] + 1) // 2, c["ctx"] + 1, n)
        most = min(w, 8)                                         # accepted tokens: a path down the tree
        keep = np.sort(np.stack([rng.permutation(w)[:most] for _ in range(n)]), 1)
        count = rng.integers(0, most + 1, n)
        row_pages = -(-(c["ctx"] + most + w) // slots)
        # a step leaves at most `most` tokens behind the base, which the next one replaces
        pages = n * row_pages + 2
        table = np.full((n, row_pages), -1, dtype=np.int32)
        order, used = rng.permutation(pages), 0
        refs = np.zeros(pages, dtype=np.int32)
        for r in range(n):
            k = -(-int(base[r]) // slots)
            table[r, :k] = order[used:used + k]
            refs[order[used:used + k]] = 1
            used += k
        s["table"], s["refs"], s["lens"] = _ints(table), _ints(refs), _ints(base)
        s["rows"] = _ints(rng.permutation(n))
        s["from"] = s["lens"][s["rows"].long()].clone()
        s["add"] = _ints(np.full(n, w))
        s["keep"], s["count"] = _ints(keep), _ints(count)
        s["grown"], s["kept"] = _ints(np.zeros(n)), _ints(np.zeros(n))
        s["pools"] = []
        for _ in range(c["pools"]):
            pool = _empty_pool(c, pages, torch.int16 if c["fmt"] == "same" else torch.uint8)
            s["pools"].append(pool.random_(0, 255, generator=g))


def _frequencies(c):
    """Angle per position of each pair, in radians."""
    n = c["rot"]
    return 10000.0 ** (-2 * np.arange(n // 2, dtype=np.float64) / n)


# ---- the library's side ----------------------------------------------------

_NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.int16: "u16", torch.uint8: "u8"}


def _map(att, t):
    """The tensor map of a torch tensor, dimensions innermost first."""
    n = t.element_size()
    dims = tuple(reversed(t.shape))
    strides = tuple(n * st for st in reversed(t.stride()[:-1]))
    return att.tmap_encode(_NAMES[t.dtype], t.dim(), t.data_ptr(), dims, strides, (16 // n,) + (1,) * (t.dim() - 1))


def _pool_map(att, t, c):
    """The map of a pool: dims (dim, rows, heads, pages)."""
    return _map(att, _heads(t, c))


class _Handles:
    @staticmethod
    def window(att, c, s):
        s["mq"], s["mo"] = _map(att, s["q"]), _map(att, s["o"])
        s["mk"], s["mv"] = (_pool_map(att, s[n], c) for n in ("k_pool", "v_pool"))
        s["pt"] = att.page_table(s["table"], s["lens"], None, s["k_pool"].shape[0], c["slots"])
        s["ws"] = torch.empty(att.attn_cache_workspace(s["mq"], s["mk"], c["window"], c["sinks"], c["ctx"]), device=DEV,
                              dtype=torch.uint8)

    tree = window

    @staticmethod
    def append(att, c, s):
        s["plan"] = att.rope_encode(c["rot"], c["layout"], 10000.0)
        s["m"] = [_map(att, s[n]) for n in ("q", "q_out", "k", "v")]
        s["back"] = [_map(att, s[n]) for n in ("k_back", "v_back")]
        s["mk"], s["mv"] = (_pool_map(att, s[n], c) for n in ("k_pool", "v_pool"))
        s["pt"] = att.page_table(s["table"], None, None, s["k_pool"].shape[0], c["slots"])

    @staticmethod
    def read(att, c, s):
        s["back"] = [_map(att, s[n]) for n in ("k", "v")]
        s["mk"], s["mv"] = (_pool_map(att, s[n], c) for n in ("k_pool", "v_pool"))
        s["pt"] = att.page_table(s["table"], None, None, c["pages"], c["slots"])

    @staticmethod
    def verify(att, c, s):
        s["pt"] = att.page_table(s["table"], s["lens"], s["refs"], s["refs"].numel(), c["slots"])
        s["maps"] = att.tmap_array([_pool_map(att, p, c) for p in s["pools"]])
        s["ws"] = torch.empty(att.page_workspace(s["pt"], c["batch"]), device=DEV, dtype=torch.uint8)


class _Own:
    @staticmethod
    def window(c, s, st):
        s["att"].attn_window(s["mq"], s["mk"], s["mv"], c["fmt"], s["pt"], s["rows"], s["count"] if c["ragged"] else None,
                             c["window"], c["sinks"], c["ctx"], s["scale"], s["mo"], s["lse"], s["ws"], st)
        return s["o"], s["lse"]

    @staticmethod
    def tree(c, s, st):
        s["att"].attn_tree(s["mq"], s["mk"], s["mv"], c["fmt"], s["pt"], s["rows"], s["count"], s["parent"], c["window"],
                           c["sinks"], c["ctx"], s["scale"], s["mo"], s["lse"], s["ws"], st)
        return s["o"], s["lse"]

    @staticmethod
    def append(c, s, st):
        q, q_out, k, v = s["m"]
        s["att"].kv8_append(s["plan"], q, q_out, k, v, c["fmt"], s["mk"], s["mv"], s["pt"], s["rows"], s["at"], s["pos"],
                            st)
        s["att"].kv8_read(c["fmt"], s["mk"], s["mv"], s["pt"], s["rows"], s["at"], *s["back"], st)
        return s["q_out"], s["k_back"], s["v_back"]

    @staticmethod
    def read(c, s, st):
        s["att"].kv8_read(c["fmt"], s["mk"], s["mv"], s["pt"], s["rows"], s["at"], *s["back"], st)
        return s["k"], s["v"]

    @staticmethod
    def verify(c, s, st):
        att, n = s["att"], c["batch"]
        att.page_extend(s["pt"], s["rows"], s["add"], n, s["grown"], s["ws"], st)
        att.page_keep(s["pt"], s["maps"], s["rows"], s["from"], s["keep"], s["count"], n, s["kept"], st)
        return s["table"], s["lens"], s["refs"], s["grown"], s["kept"], s["pools"]


# ---- the plain forms -------------------------------------------------------

def _rotate(x, pos, freq, layout):
    """x [tokens, heads, dim] rotated over its first 2 * len(freq) elements, in fp32."""
    n = 2 * freq.numel()
    a = pos.double()[:, None] * freq
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    f = x.float()
    r = f[..., :n]
    u, v = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :n // 2], r[..., n // 2:])
    p, q = u * cos - v * sin, u * sin + v * cos
    r = torch.stack((p, q), -1).flatten(-2) if layout == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((r, f[..., n:]), -1)


def _scale_bytes(c, slot):
    """Row and columns of the scales of `slot` in a head of an 8-bit page."""
    at = 2 * slot
    return c["slots"] + at // c["dim"], (at % c["dim"])[..., None] + torch.arange(2, device=DEV)


def _gather(pool, c, page, slot):
    """Tokens (page, slot) of a pool, [..., heads, dim] in fp32."""
    heads = _heads(pool, c)
    x = heads[page, :, slot]
    if c["fmt"] == "same":
        return x.float()
    row, col = _scale_bytes(c, slot)
    scale = heads[page[..., None], :, row[..., None], col]       # [..., 2, heads]
    scale = scale.transpose(-1, -2).flatten().view(torch.bfloat16).view(x.shape[:-1] + (1,))
    x = x.view(torch.int8) if c["fmt"] == "int8" else x.view(torch.float8_e4m3fn)
    return x.float() * scale.float()


class _Plain:
    @staticmethod
    def window(c, s, depth=None, related=None):
        batch, n_q, kv, dim, slots, heads = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["slots"], c["heads"]
        group, held, count = heads // kv, s["lens"].long()[s["rows"].long()], s["count"].long()
        first = held - count                                     # position of each sequence's first query
        j = torch.arange(n_q, device=DEV)
        here = j if depth is None else depth                     # [n_q] or [batch, n_q]: positions from there on
        at = (first[:, None] + here)[..., None]
        # the tokens that any query of a sequence may see: the first few, and those up to the window's reach
        span, few = c["ctx"], 0
        if c["window"] and c["window"] + n_q + c["sinks"] < c["ctx"]:
            span, few = c["window"] + n_q, c["sinks"]
        low = (held - span).clamp(min=0)[:, None]
        t = torch.cat((torch.arange(few, device=DEV).expand(batch, few), low + torch.arange(span, device=DEV)), 1)
        whole = torch.cat((torch.arange(few, device=DEV) < low, torch.ones((batch, span), dtype=torch.bool, device=DEV)), 1)
        whole = whole & (t < held[:, None])
        page = s["table"][s["rows"].long()].long().gather(1, (t // slots).clamp(max=s["table"].shape[1] - 1))
        k, v = (_gather(s[p], c, page, t % slots) for p in ("k_pool", "v_pool"))
        k, v = (x.permute(0, 2, 1, 3).reshape(batch * kv, t.shape[1], dim) for x in (k, v))
        tok = t[:, None]
        if related is None:
            where, seen = tok, tok <= at
        else:  # drafted tokens stand where their depth says
            node = tok - first[:, None, None]
            drafted = node >= 0
            nodes = node.clamp(0, n_q - 1)
            where = torch.where(drafted, first[:, None, None] + depth[:, None].gather(2, nodes), tok)
            seen = ~drafted | related.gather(2, nodes.expand(batch, n_q, -1))
        if c["window"]:
            seen = seen & ((where > at - c["window"]) | (where < c["sinks"]))
        seen = (seen & whole[:, None])[:, None, :, None]
        q = s["q"].float().view(batch, n_q, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch * kv, n_q * group, dim)
        a = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(s["scale"]).view(batch, kv, n_q, group, -1)
        a.masked_fill_(~seen, -math.inf)
        top = a.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        a.sub_(top).exp_()
        total = a.sum(-1, keepdim=True)
        o = torch.bmm(a.view(batch * kv, n_q * group, -1), v).view(batch, kv, n_q, group, dim)
        o = torch.where(total > 0, o / total, 0.0)
        lse = top + total.log()

        def back(x):
            return x.permute(0, 2, 1, 3, 4).reshape(batch, n_q, heads, -1)

        asked = (j < count[:, None])[..., None]
        s["o"] = torch.where(asked[..., None], back(o).to(s["q"].dtype), s["o"])
        s["lse"] = torch.where(asked, back(lse)[..., 0], s["lse"])
        return s["o"], s["lse"]

    @staticmethod
    def tree(c, s):
        n = c["q_len"]
        parent = s["parent"].long()
        up = torch.eye(n, device=DEV) + (parent[..., None] == torch.arange(n, device=DEV)).float()
        for _ in range(max(1, (n - 1).bit_length())):            # each time twice as far up
            up = (torch.bmm(up, up) > 0).float()
        related = up > 0
        return _Plain.window(c, s, related.sum(-1) - 1, related)

    @staticmethod
    def append(c, s):
        at, rows = s["at"].long(), s["rows"].long()
        page, slot = s["table"][rows, at // c["slots"]].long(), at % c["slots"]
        k = _rotate(s["k"], s["pos"], s["freq"], c["layout"])
        back = [_Plain._store(c, s[p], page, slot, x) for p, x in (("k_pool", k), ("v_pool", s["v"].float()))]
        q = _rotate(s["q"], s["pos"], s["freq"], c["layout"]).to(s["q"].dtype)
        return (q, *(x.to(s["k"].dtype) for x in back))

    @staticmethod
    def _store(c, pool, page, slot, x):
        scale = _scale(x, TOP[c["fmt"]])
        # in 64 bits: many values of a few bits lie on the border between two codes
        y = torch.where(scale > 0, x.double() / scale.double(), 0.0).float().clamp(-TOP[c["fmt"]], TOP[c["fmt"]])
        code = y.round().to(torch.int8) if c["fmt"] == "int8" else y.to(torch.float8_e4m3fn)
        heads = _heads(pool, c)
        heads[page, :, slot] = code.view(torch.uint8)
        row, col = _scale_bytes(c, slot)
        heads[page[..., None], :, row[..., None], col] = scale.flatten().view(torch.uint8).view(
            scale.shape[:-1] + (2,)).transpose(-1, -2)
        return _gather(pool, c, page, slot)

    @staticmethod
    def read(c, s):
        at = s["at"].long()
        page, slot = s["table"][0][at // c["slots"]].long(), at % c["slots"]
        return tuple(_gather(s[p], c, page, slot).to(TYPES[c["dtype"]]) for p in ("k_pool", "v_pool"))

    @staticmethod
    def verify(c, s):
        table, lens, refs, slots, rows = s["table"], s["lens"], s["refs"], c["slots"], s["rows"].long()
        n, col = table.shape[1], torch.arange(table.shape[1], device=DEV)
        # the rows grow by their drafted tokens: the free pages of lowest index, handed out in order
        held = lens[rows]
        start, end = -(-held // slots), -(-(held + s["add"]) // slots)
        busy = refs > 0
        free, pages = (~busy).sum(), torch.sort(busy.to(torch.int8), stable=True).indices
        rank = (end - start).cumsum(0)
        grown = (rank <= free) & (end <= n)
        fresh = (col >= start[:, None]) & (col < end[:, None]) & grown[:, None]
        which = (rank - (end - start))[:, None] + col - start[:, None]
        more = pages[which.clamp(0, refs.numel() - 1)]
        table[rows] = torch.where(fresh, more.int(), table[rows])
        refs.index_add_(0, more.flatten(), fresh.flatten().int())
        held = torch.where(grown, held + s["add"], held)
        # the accepted tokens move together
        width = s["keep"].shape[1]
        w, count, first = torch.arange(width, device=DEV), s["count"], s["from"]
        last = s["keep"].gather(1, (count - 1).clamp(min=0)[:, None].long())[:, 0]
        kept = (first + torch.where(count > 0, last + 1, 0)) <= held
        pairs = (kept[:, None] & (w < count[:, None])).nonzero()
        i, j = pairs[:, 0], pairs[:, 1]
        src, dst, row = (first[i] + s["keep"][i, j]).long(), (first[i] + j).long(), rows[i]
        src_page, dst_page = table[row, src // slots].long(), table[row, dst // slots].long()
        src, dst = src % slots, dst % slots
        for p in s["pools"]:
            h = _heads(p, c)
            old = h[src_page, :, src]
            if c["fmt"] != "same":
                row, byte = _scale_bytes(c, src)
                scale = h[src_page[:, None], :, row[:, None], byte]
                row, byte = _scale_bytes(c, dst)
                h[dst_page[:, None], :, row[:, None], byte] = scale
            h[dst_page, :, dst] = old
        # the rest is dropped, pages with no token left are given back
        left = torch.where(kept, first + count, held)
        gone = (col >= -(-left // slots)[:, None]) & (table[rows] >= 0)
        old = table[rows].clamp(min=0).long()
        refs.index_add_(0, old.flatten(), -gone.flatten().int())
        table[rows] = torch.where(gone, -1, table[rows])
        lens[rows] = left
        return table, lens, refs, grown.int(), kept.int(), s["pools"]


def run(state):
    c = state["case"]
    if own:
        return getattr(_Own, c["op"])(c, state, torch.cuda.current_stream().cuda_stream)
    return getattr(_Plain, c["op"])(c, state)


# ---- what a pass cannot do without -----------------------------------------

_SIZES = {"f16": 2, "bf16": 2, "f32": 4}


def work(case):
    c = case
    if c["op"] in ("window", "tree"):
        e = _SIZES[c["dtype"]]
        token = 2 * c["kv_heads"] * (c["dim"] * e if c["fmt"] == "same" else c["dim"] + 2)
        tokens = pairs = asked = 0
        for held, n in zip(_held(c), _counts(c)):
            first = held - n
            asked += n
            if c["op"] == "tree":  # the context, and of the drafted tokens those on the way to each
                reach = min(first, c["window"] + c["sinks"]) if c["window"] else first
                tokens += reach + n
                pairs += n * (reach + 4)
                continue
            p = np.arange(first, held)[np.arange(first, held) >= 0]
            seen = p + 1
            if c["window"]:
                seen = np.minimum(seen, c["window"]) + np.minimum(c["sinks"], np.maximum(p + 1 - c["window"], 0))
            pairs += int(seen.sum())
            tokens += min(held, c["window"] + n - 1 + c["sinks"]) if c["window"] else held
        return {"bytes": tokens * token + asked * c["heads"] * (2 * c["dim"] * e + 4),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "append":
        e, n = _SIZES[c["dtype"]], c["tokens"]
        written = 2 * c["kv_heads"] * (c["dim"] + 2)
        return {"bytes": n * ((2 * c["heads"] + 4 * c["kv_heads"]) * c["dim"] * e + 2 * written + 12),
                "flops": n * (3 * (c["heads"] + c["kv_heads"]) * c["rot"] + 6 * c["kv_heads"] * c["dim"])}
    if c["op"] == "read":
        return {"bytes": c["tokens"] * (2 * c["kv_heads"] * ((1 + _SIZES[c["dtype"]]) * c["dim"] + 2) + 8),
                "flops": 2 * c["tokens"] * c["kv_heads"] * c["dim"]}
    token = c["kv_heads"] * (2 * c["dim"] if c["fmt"] == "same" else c["dim"] + 2)
    entries = c["batch"] * (2 + c["nodes"] / c["slots"])
    return {"bytes": c["batch"] * (min(c["nodes"], 8) / 2 * 2 * token * c["pools"] + 64) + 24 * entries, "flops": 0}


# ---- the definitions in 64 bits --------------------------------------------

def _values(pool, c, page):
    """Pages of a pool as [len(page) * slots, heads, dim] in 64 bits."""
    x = pool[page]
    x = x.transpose(1, 2) if c["heads_first"] else x             # [n, rows, heads, dim]
    if c["fmt"] == "same":
        return x.double().flatten(0, 1)
    code, tail = x[:, :c["slots"]], x[:, c["slots"]:]
    tail = tail.permute(0, 2, 1, 3).flatten().view(torch.bfloat16).view(x.shape[0], c["kv_heads"], -1)
    tail = tail[..., :c["slots"]].permute(0, 2, 1)[..., None].double()
    code = code.contiguous().view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn).double()
    return (code * tail).flatten(0, 1)


def _turned(x, pos, c):
    """Each pair of x as a complex number times exp(i * pos * frequency), in 64 bits."""
    n = c["rot"]
    theta = torch.tensor([math.exp(-2.0 * j / n * math.log(10000.0)) for j in range(n // 2)], dtype=torch.float64,
                         device=x.device)
    turn = pos.double()[:, None] * theta
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    y = x.double().clone()
    first, second = (slice(0, n, 2), slice(1, n, 2)) if c["layout"] == "interleaved" else (slice(0, n // 2),
                                                                                          slice(n // 2, n))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _as_8_bits(y, fmt):
    """The values that 8 bits and one scale a head leave of y.  The scale has eight significant bits, rounded up."""
    scale = y.abs().amax(-1, keepdim=True) / TOP[fmt]
    step = torch.exp2(torch.floor(torch.log2(scale)) - 7)
    scale = torch.ceil(scale / step) * step
    z = y / scale
    if fmt == "int8":
        z = torch.round(z)
    else:  # four significant bits, down to steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        z = torch.round(z / step) * step
    return torch.where(scale > 0, z * scale, 0.0)


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None  # whole numbers alone
    s = {"case": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    getattr(_Inputs, c["op"])(c, g, np.random.default_rng(seed), s)
    if c["op"] == "append":
        return _turned(s["q"], s["pos"], c), _as_8_bits(_turned(s["k"], s["pos"], c), c["fmt"]), \
            _as_8_bits(s["v"].double(), c["fmt"])
    if c["op"] == "read":
        at = s["at"].long()
        page = s["table"][0].long()
        return tuple(_values(s[p], c, page)[at] for p in ("k_pool", "v_pool"))
    # attention, one sequence and one shared head after the other
    n_q, kv = c["q_len"], c["kv_heads"]
    group = c["heads"] // kv
    rows, lens, counts = (s[x].cpu().tolist() for x in ("rows", "lens", "count"))
    parents = s["parent"].cpu().tolist() if c["op"] == "tree" else None
    out, lse = s["o"].double(), s["lse"].double()
    for b in range(c["batch"]):
        n, held = counts[b], lens[rows[b]]
        first = held - n
        if n == 0:
            continue
        see = np.zeros((n, held), dtype=bool)
        t = np.arange(held)
        for j in range(n):
            if parents is None:
                p = first + j
                see[j] = (t <= p) & ((t > p - c["window"]) | (t < c["sinks"]) if c["window"] else True)
                continue
            way = [j]
            while parents[b][way[-1]] >= 0:
                way.append(parents[b][way[-1]])
            place = dict((node, first + len(way) - 1 - i) for i, node in enumerate(way))
            p = place[j]
            see[j, :first] = (t[:first] > p - c["window"]) | (t[:first] < c["sinks"]) if c["window"] else True
            for node, at in place.items():
                see[j, first + node] = not c["window"] or at > p - c["window"] or at < c["sinks"]
        see = torch.from_numpy(see).to(DEV)
        if held == 0:
            out[b, :n], lse[b, :n] = 0.0, -math.inf
            continue
        page = s["table"][rows[b], :-(-held // c["slots"])].long()
        k, v = (_values(s[p], c, page)[:held].transpose(0, 1).contiguous() for p in ("k_pool", "v_pool"))
        for h in range(kv):
            for i in range(group):
                q = s["q"][b, :n, h * group + i].double()
                score = (q @ k[h].t().contiguous() * s["scale"]).masked_fill(~see, -math.inf)
                total = torch.logsumexp(score, -1)
                empty = total == -math.inf
                w = torch.exp(score - torch.where(empty, 0.0, total)[:, None])
                out[b, :n, h * group + i], lse[b, :n, h * group + i] = w @ v[h], total
    return out, lse
