"""The cache operators' measured cases: what each computes, in plain torch and
through the library, and what it cannot do without.

Five operators of a paged key / value cache, on the sizes real serving meets:

``rope``     rotary positions on a tensor of heads (forward, and its gradient,
             which is the rotation by the negative angle)
``append``   one step's queries and keys rotated, keys and values written to
             their pages
``fork``     one sampling step's bookkeeping: rows given back, forked from
             their parents (shared pages counted, the unfinished page copied)
             and extended by their next tokens
``compact``  the pages in use moved to the lowest indices, tables rewritten
``attn``     attention of a batch whose sequences share a long prefix

A pool of pages is a tensor [pages, slots, heads, dim] or, where a case says
``heads_first``, [pages, heads, slots, dim].  Page tables, lengths and
reference counts are int32.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases -------------------------------------------------------------

def listed():
    return [
        # eight sequences' next token: the smallest call, half of each head rotated in pairs
        dict(name="rope decode bf16 pairs", op="rope", dtype="bf16", tokens=8, heads=16, dim=128, rot=64,
             layout="interleaved", scaling="none", factor=1.0, magnitude=1.0, far=4096, inverse=False),
        # a long prompt at positions past the trained length, frequencies scaled by parts
        dict(name="rope prompt bf16 far", op="rope", dtype="bf16", tokens=8192, heads=32, dim=128, rot=128,
             layout="half", scaling="ramp", factor=16.0, magnitude=1.2, far=1 << 20, inverse=False),
        # a training step's gradient in fp32, odd token count, the base scaled
        dict(name="rope gradient f32", op="rope", dtype="f32", tokens=4095, heads=24, dim=96, rot=96,
             layout="half", scaling="base", factor=4.0, magnitude=1.0, far=32768, inverse=True),
        # 64 sequences' next token written to its page
        dict(name="append decode f16", op="append", dtype="f16", tokens=64, rows=64, heads=32, kv_heads=8, dim=128,
             rot=128, layout="half", slots=16, row_tokens=2048, heads_first=False),
        # a chunk of several prompts, pages of an odd size, heads outermost in the page
        dict(name="append prompt bf16", op="append", dtype="bf16", tokens=8191, rows=5, heads=32, kv_heads=8, dim=128,
             rot=96, layout="interleaved", slots=48, row_tokens=4096, heads_first=True),
        # four continuations of one sequence, two layers' keys and values
        dict(name="fork 4 of 1", op="fork", pages=1024, slots=16, heads=8, dim=128, pools=4, parents=1, children=4,
             row_tokens=512, add=1),
        # a wide sampling step over many sequences, eight layers
        dict(name="fork 128 of 48", op="fork", pages=16384, slots=16, heads=4, dim=128, pools=16, parents=48,
             children=128, row_tokens=4096, add=5),
        # a small pool after a few sequences ended
        dict(name="compact 500 pages", op="compact", pages=500, slots=16, heads=8, dim=64, pools=2, rows=16,
             row_tokens=256, used=0.6),
        # a large pool, half of it given back in scattered order
        dict(name="compact 16384 pages", op="compact", pages=16384, slots=16, heads=4, dim=128, pools=8, rows=64,
             row_tokens=4096, used=0.5),
        # four short answers behind one system prompt: latency counts
        dict(name="attn 4 x 512+32 f16", op="attn", dtype="f16", batch=4, q_len=1, heads=8, kv_heads=2, dim=64,
             slots=16, prefix=512, suffix=32, heads_first=False),
        # drafted tokens checked three at a time, pages of an odd size
        dict(name="attn 32 x 8192+1000 q3 bf16", op="attn", dtype="bf16", batch=32, q_len=3, heads=32, kv_heads=8,
             dim=128, slots=48, prefix=8192, suffix=1000, heads_first=True),
        # a large batch over one long document
        dict(name="attn 128 x 32768+1024 bf16", op="attn", dtype="bf16", batch=128, q_len=1, heads=32, kv_heads=8,
             dim=128, slots=16, prefix=32768, suffix=1024, heads_first=False),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append", "fork", "compact", "attn"])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    slots = rng.choice([1, 8, 16, 32, 48, 64, 100, 256])
    if op == "rope":
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), tokens=_between(rng, 1, 4096),
                    heads=_between(rng, 1, 32), dim=dim, rot=2 * rng.randint(1, dim // 2),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "ramp"]), factor=rng.choice([2.0, 4.0, 10.0]),
                    magnitude=rng.choice([1.0, 1.1]), far=_between(rng, 64, 1 << 22), inverse=rng.random() < 0.5)
    if op == "append":
        kv = rng.choice([1, 2, 4, 8])
        rows = _between(rng, 1, 64)
        tokens = _between(rng, rows, 4096)
        return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), tokens=tokens, rows=rows,
                    heads=kv * rng.randint(1, 4), kv_heads=kv, dim=dim, rot=2 * rng.randint(1, dim // 2),
                    layout=rng.choice(["half", "interleaved"]), slots=slots,
                    row_tokens=-(-tokens // rows) + _between(rng, 1, 512), heads_first=rng.random() < 0.5)
    if op == "fork":
        slots = rng.choice([8, 16, 32, 48, 64])
        parents, children = _between(rng, 1, 48), _between(rng, 1, 128)
        row_tokens = _between(rng, 1, 2048)
        row_pages = -(-row_tokens // slots)
        add = rng.randint(0, 40)
        need = parents * row_pages + children * (2 + add // slots)
        return dict(op=op, pages=need + rng.randint(-min(need // 8, children), need // 4), slots=slots,
                    heads=rng.choice([1, 2, 4]), dim=rng.choice([64, 80, 128]), pools=rng.choice([1, 2, 3, 8]),
                    parents=parents, children=children, row_tokens=row_tokens, add=add)
    if op == "compact":
        slots = rng.choice([1, 8, 16, 48])
        return dict(op=op, pages=_between(rng, 1, 8192), slots=slots, heads=rng.choice([1, 2, 4]),
                    dim=rng.choice([64, 80, 128]), pools=rng.choice([1, 2, 5]), rows=_between(rng, 1, 64),
                    row_tokens=slots * _between(rng, 1, 128), used=rng.choice([0.0, 0.1, 0.5, 0.9, 1.0]))
    kv = rng.choice([1, 2, 4, 8])
    return dict(op=op, dtype=rng.choice(["f16", "bf16"]), batch=_between(rng, 1, 64), q_len=rng.choice([1, 1, 2, 5]),
                heads=kv * rng.choice([1, 2, 4, 5]), kv_heads=kv, dim=dim, slots=slots,
                prefix=rng.choice([0, _between(rng, 1, 16384), _between(rng, 1, 16384)]),
                suffix=_between(rng, 1, 1024), heads_first=rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).to(DEV)


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
    def rope(c, g, rng, s):
        s["x"] = _normal(g, (c["tokens"], c["heads"], c["dim"]), TYPES[c["dtype"]])
        s["y"] = torch.empty_like(s["x"])
        s["pos"] = _ints(rng.integers(0, c["far"], c["tokens"]))
        s["freq"] = torch.from_numpy(_frequencies(c)).to(DEV)

    @staticmethod
    def append(c, g, rng, s):
        t, n, r = TYPES[c["dtype"]], c["tokens"], c["rows"]
        s["q"] = _normal(g, (n, c["heads"], c["dim"]), t)
        s["q_out"] = torch.empty_like(s["q"])
        s["k"] = _normal(g, (n, c["kv_heads"], c["dim"]), t)
        s["v"] = _normal(g, (n, c["kv_heads"], c["dim"]), t)
        row_pages = -(-c["row_tokens"] // c["slots"])
        pages = r * row_pages
        s["k_pool"] = _pool(g, c, pages, t)
        s["v_pool"] = _pool(g, c, pages, t)
        s["table"] = _ints(rng.permutation(pages).reshape(r, row_pages))
        # each row's next tokens, after what it holds; rows differ by at most one token
        per = np.bincount(np.arange(n) % r, minlength=r)
        held = [int(rng.integers(0, c["row_tokens"] - p + 1)) for p in per]
        s["rows"] = _ints(np.repeat(np.arange(r), per))
        s["at"] = _ints(np.concatenate([h + np.arange(p) for h, p in zip(held, per)]))
        s["pos"] = s["at"] + int(rng.integers(0, 1 << 16))  # behind a prefix of that length
        s["freq"] = torch.from_numpy(_frequencies(c)).to(DEV)

    @staticmethod
    def fork(c, g, rng, s):
        parents, children, slots = c["parents"], c["children"], c["slots"]
        held = rng.integers(1, c["row_tokens"] + 1, parents)
        row_pages = -(-(c["row_tokens"] + c["add"]) // slots)
        table = np.full((parents + children, row_pages), -1, dtype=np.int32)
        order = rng.permutation(c["pages"])
        used = 0
        for p in range(parents):
            k = -(-int(held[p]) // slots)
            if used + k > c["pages"]:
                held[p], k = 0, 0
            table[p, :k] = order[used:used + k]
            used += k
        refs = np.zeros(c["pages"], dtype=np.int32)
        refs[order[:used]] = 1
        s["table"], s["refs"] = _ints(table), _ints(refs)
        s["lens"] = _ints(np.concatenate([held, np.zeros(children)]))
        s["from"] = _ints(rng.integers(0, parents, children))
        s["to"] = _ints(parents + rng.permutation(children))
        s["add"] = _ints(rng.integers(0, c["add"] + 1, children))
        s["forked"], s["grown"] = _ints(np.zeros(children)), _ints(np.zeros(children))
        s["pools"] = [_bits(g, c) for _ in range(c["pools"])]

    @staticmethod
    def compact(c, g, rng, s):
        row_pages = -(-c["row_tokens"] // c["slots"])
        want = min(int(c["used"] * c["pages"]), c["rows"] * row_pages)
        table = np.full((c["rows"], row_pages), -1, dtype=np.int32)
        held = np.zeros(c["rows"], dtype=np.int32)
        order = rng.permutation(c["pages"])[:want]
        part = np.zeros(c["rows"], dtype=np.int64)  # how many pages each row holds: all of `want`, at random
        left = want
        for r in rng.permutation(c["rows"]):
            part[r] = min(left, row_pages, int(math.ceil(2 * want / c["rows"] * rng.random())))
            left -= part[r]
        for r in range(c["rows"]):
            more = min(left, row_pages - int(part[r]))
            part[r] += more
            left -= more
        at = 0
        refs = np.zeros(c["pages"], dtype=np.int32)
        for r in range(c["rows"]):
            k = int(part[r])
            table[r, :k] = order[at:at + k]
            refs[order[at:at + k]] += 1
            held[r] = 0 if k == 0 else (k - 1) * c["slots"] + int(rng.integers(1, c["slots"] + 1))
            at += k
        if c["rows"] > 1:  # two rows share the pages of the first
            refs[table[0][table[0] >= 0]] += 1
            old = table[1][table[1] >= 0]
            refs[old] -= 1
            table[1], held[1] = table[0], held[0]
        s["table"], s["refs"], s["lens"] = _ints(table), _ints(refs), _ints(held)
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["used"] = _ints([0])
        s["pools"] = [_bits(g, c) for _ in range(c["pools"])]

    @staticmethod
    def attn(c, g, rng, s):
        t, slots = TYPES[c["dtype"]], c["slots"]
        s["q"] = _normal(g, (c["batch"], c["q_len"], c["heads"], c["dim"]), t)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["batch"], c["q_len"], c["heads"]), device=DEV, dtype=torch.float32)
        shared, each = -(-c["prefix"] // slots), -(-c["suffix"] // slots)
        pages = shared + c["batch"] * each + 3
        s["k_pool"], s["v_pool"] = _pool(g, c, pages, t), _pool(g, c, pages, t)
        order = rng.permutation(pages)
        # row 0 is the prefix's; the rows of the batch follow
        table = np.full((c["batch"] + 1, max(shared, each, 1)), -1, dtype=np.int32)
        table[0, :shared] = order[:shared]
        table[1:, :each] = order[shared:shared + c["batch"] * each].reshape(c["batch"], each)
        held = rng.integers(0, c["suffix"] + 1, c["batch"] + 1)
        held[0], held[1], held[-1] = c["prefix"], c["suffix"], 0 if c["batch"] > 1 else c["suffix"]
        s["table"], s["lens"] = _ints(table), _ints(held)
        s["rows"] = _ints(1 + np.arange(c["batch"]))
        s["scale"] = 1.0 / math.sqrt(c["dim"])


def _pool(g, c, pages, t):
    a, b = (c["kv_heads"], c["slots"]) if c["heads_first"] else (c["slots"], c["kv_heads"])
    return _normal(g, (pages, a, b, c["dim"]), t)


def _bits(g, c):
    return torch.randint(-32768, 32768, (c["pages"], c["slots"], c["heads"], c["dim"]), generator=g, device=DEV,
                         dtype=torch.int16)


def _frequencies(c):
    """Angle per position of each pair, in radians."""
    n = c["rot"]
    j = np.arange(n // 2, dtype=np.float64)
    base, scaling, factor = 10000.0, c.get("scaling", "none"), c.get("factor", 1.0)
    if scaling == "base" and n > 2:
        base *= factor ** (n / (n - 2))
    f = base ** (-2 * j / n)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":  # frequencies of many turns over 4096 positions stay, those of few are stretched
        w = np.clip((4096 * f / (2 * np.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * (w + (1 - w) / factor)
    return f


# ---- the library's side ----------------------------------------------------

_NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.int16: "u16"}


def _map(att, t):
    """The tensor map of a torch tensor, dimensions innermost first."""
    n = t.element_size()
    vec = 16 // n
    dims = tuple(reversed(t.shape))
    strides = tuple(n * st for st in reversed(t.stride()[:-1]))
    return att.tmap_encode(_NAMES[t.dtype], t.dim(), t.data_ptr(), dims, strides, (vec,) + (1,) * (t.dim() - 1))


def _pool_map(att, t, heads_first):
    """The map of a pool: dims (dim, slots, heads, pages)."""
    return _map(att, t if heads_first else t.transpose(1, 2))


def _plan(att, c):
    return att.rope_encode(c["rot"], c["layout"], 10000.0, c.get("scaling", "none"), c.get("factor", 1.0), 4096, 1.0,
                           32.0, c.get("magnitude", 1.0))


class _Handles:
    @staticmethod
    def rope(att, c, s):
        s["plan"], s["mx"], s["my"] = _plan(att, c), _map(att, s["x"]), _map(att, s["y"])

    @staticmethod
    def append(att, c, s):
        s["plan"] = _plan(att, c)
        s["m"] = [_map(att, s[n]) for n in ("q", "q_out", "k", "v")]
        s["m"] += [_pool_map(att, s[n], c["heads_first"]) for n in ("k_pool", "v_pool")]
        s["pt"] = att.page_table(s["table"], None, None, s["k_pool"].shape[0], c["slots"])

    @staticmethod
    def fork(att, c, s):
        s["pt"] = att.page_table(s["table"], s["lens"], s["refs"], c["pages"], c["slots"])
        s["maps"] = att.tmap_array([_pool_map(att, p, False) for p in s["pools"]])
        s["ws"] = torch.empty(att.page_workspace(s["pt"], c["children"]), device=DEV, dtype=torch.uint8)

    @staticmethod
    def compact(att, c, s):
        s["pt"] = att.page_table(s["table"], s["lens"], s["refs"], c["pages"], c["slots"])
        s["pt_out"] = att.page_table(s["table_out"], s["lens"], s["refs_out"], c["pages"], c["slots"])
        s["maps"] = att.tmap_array([_pool_map(att, p, False) for p in s["pools"]])
        s["ws"] = torch.empty(att.page_workspace(s["pt"], 0), device=DEV, dtype=torch.uint8)

    @staticmethod
    def attn(att, c, s):
        s["mq"], s["mo"] = _map(att, s["q"]), _map(att, s["o"])
        s["mk"], s["mv"] = (_pool_map(att, s[n], c["heads_first"]) for n in ("k_pool", "v_pool"))
        s["pt"] = att.page_table(s["table"], s["lens"], None, s["k_pool"].shape[0], c["slots"])
        s["ws"] = torch.empty(att.attn_workspace(s["mq"], s["mk"], c["prefix"], c["suffix"]), device=DEV,
                              dtype=torch.uint8)


class _Own:
    @staticmethod
    def rope(c, s, st):
        s["att"].rope_apply(s["plan"], s["mx"], s["my"], s["pos"], c["inverse"], st)
        return s["y"]

    @staticmethod
    def append(c, s, st):
        q, q_out, k, v, k_pool, v_pool = s["m"]
        s["att"].rope_append(s["plan"], q, q_out, k, v, k_pool, v_pool, s["pt"], s["rows"], s["at"], s["pos"], st)
        return s["q_out"], s["k_pool"], s["v_pool"]

    @staticmethod
    def fork(c, s, st):
        att, n = s["att"], c["children"]
        att.page_free(s["pt"], s["to"], n, st)
        att.page_fork(s["pt"], s["maps"], s["from"], s["to"], n, s["forked"], s["ws"], st)
        att.page_extend(s["pt"], s["to"], s["add"], n, s["grown"], s["ws"], st)
        return s["table"], s["lens"], s["refs"], s["forked"], s["grown"], s["pools"]

    @staticmethod
    def compact(c, s, st):
        s["att"].page_compact(s["pt"], s["pt_out"], s["maps"], s["used"], s["ws"], st)
        return s["table_out"], s["refs_out"], s["used"], s["pools"]

    @staticmethod
    def attn(c, s, st):
        s["att"].attn_shared_prefix(s["mq"], s["mk"], s["mv"], s["pt"], 0, c["prefix"], s["rows"], c["suffix"],
                                    s["scale"], s["mo"], s["lse"], s["ws"], st)
        return s["o"], s["lse"]


# ---- the plain forms -------------------------------------------------------

def _rotate(x, pos, freq, layout, magnitude, sign):
    """x [tokens, heads, dim] rotated over its first 2 * len(freq) elements."""
    n = 2 * freq.numel()
    a = pos.double()[:, None] * freq
    cos, sin = (a.cos() * magnitude).float()[:, None], (a.sin() * (sign * magnitude)).float()[:, None]
    f = x.float()
    r = f[..., :n]
    u, v = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :n // 2], r[..., n // 2:])
    p, q = u * cos - v * sin, u * sin + v * cos
    r = torch.stack((p, q), -1).flatten(-2) if layout == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((r, f[..., n:]), -1).to(x.dtype)


def _first_free(refs):
    """The pages with the free ones first, lowest index first, and how many are free."""
    busy = refs > 0
    return torch.sort(busy.to(torch.int8), stable=True).indices, (~busy).sum()


class _Plain:
    @staticmethod
    def rope(c, s):
        return _rotate(s["x"], s["pos"], s["freq"], c["layout"], c["magnitude"], -1.0 if c["inverse"] else 1.0)

    @staticmethod
    def append(c, s):
        at, rows = s["at"].long(), s["rows"].long()
        page, slot = s["table"][rows, at // c["slots"]].long(), at % c["slots"]
        k = _rotate(s["k"], s["pos"], s["freq"], c["layout"], 1.0, 1.0)
        if c["heads_first"]:
            s["k_pool"][page, :, slot], s["v_pool"][page, :, slot] = k, s["v"]
        else:
            s["k_pool"][page, slot], s["v_pool"][page, slot] = k, s["v"]
        return _rotate(s["q"], s["pos"], s["freq"], c["layout"], 1.0, 1.0), s["k_pool"], s["v_pool"]

    @staticmethod
    def fork(c, s):
        table, lens, refs, slots = s["table"], s["lens"], s["refs"], c["slots"]
        to, col = s["to"].long(), torch.arange(table.shape[1], device=DEV)
        # give the rows' pages back
        old = table[to].flatten().long()
        refs.index_add_(0, old.clamp(min=0), -(old >= 0).int())
        table[to], lens[to] = -1, 0
        # share the parents' full pages; the unfinished one gets a page of its own
        src = s["from"].long()
        held = lens[src]
        full, tail = held // slots, (held % slots > 0)
        pages, free = _first_free(refs)
        rank = tail.int().cumsum(0)
        done = rank <= free
        own_page = pages[(rank - 1).clamp(0, refs.numel() - 1)]
        take = tail & done
        rows = table[src]
        at = full.clamp(max=table.shape[1] - 1).long()[:, None]
        last = rows.gather(1, at)[:, 0].long()
        some = take.nonzero()[:, 0]
        goal, last = own_page[some], last[some]
        new = torch.where(col < full[:, None], rows, -1)
        new = torch.where((col == full[:, None]) & take[:, None], own_page[:, None].int(), new)
        new = torch.where(done[:, None], new, -1)
        shared = (torch.where(col < full[:, None], rows, -1) >= 0) & done[:, None]
        refs.index_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
        refs[goal] = 1
        table[to], lens[to] = new, torch.where(done, held, 0)
        for p in s["pools"]:
            p[goal] = p[last]
        # extend the new rows by their next tokens
        held = lens[to]
        first, end = -(-held // slots), -(-(held + s["add"]) // slots)
        pages, free = _first_free(refs)
        rank = (end - first).cumsum(0)
        grown = (rank <= free) & (end <= table.shape[1])
        rows = table[to]
        fresh = (col >= first[:, None]) & (col < end[:, None]) & grown[:, None]
        which = (rank - (end - first))[:, None] + col - first[:, None]
        more = pages[which.clamp(0, refs.numel() - 1)]
        table[to] = torch.where(fresh, more.int(), rows)
        refs.index_add_(0, more.flatten(), fresh.flatten().int())
        lens[to] = torch.where(grown, held + s["add"], held)
        return table, lens, refs, done.int(), grown.int(), s["pools"]

    @staticmethod
    def compact(c, s):
        refs, table = s["refs"], s["table"]
        busy = refs > 0
        used = busy.sum()
        index = torch.arange(refs.numel(), device=DEV)
        hole = (~busy & (index < used)).nonzero()[:, 0]
        move = (busy & (index >= used)).nonzero()[:, 0]
        place = index.clone()
        place[move] = hole
        out, counts = torch.where(table >= 0, place[table.clamp(min=0).long()].int(), -1), refs.clone()
        counts[hole], counts[move] = refs[move], 0
        for p in s["pools"]:
            p[hole] = p[move]
        return out, counts, used.int()[None], s["pools"]

    @staticmethod
    def attn(c, s):
        batch, n_q, kv, dim, slots = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["slots"]
        group, prefix, suffix = c["heads"] // kv, c["prefix"], c["suffix"]
        table, held = s["table"].long(), s["lens"][1:].long()

        def tokens(pool, rows, count):  # [rows, kv, count, dim] of the rows' first tokens
            t = torch.arange(count, device=DEV)
            page, slot = rows[:, t // slots].clamp(min=0), t % slots
            got = pool[page, :, slot] if c["heads_first"] else pool[page, slot]
            return got.transpose(1, 2).float().contiguous()

        # [kv, batch, n_q * group, dim]
        q = s["q"].float().view(batch, n_q, kv, group, dim).permute(2, 0, 1, 3, 4).reshape(kv, batch, n_q * group, dim)
        flat = q.reshape(kv, -1, dim)
        k, v = tokens(s["k_pool"], table[:1], prefix)[0], tokens(s["v_pool"], table[:1], prefix)[0]
        a = (torch.bmm(flat, k.transpose(1, 2).contiguous()) * s["scale"]).view(kv, batch, n_q * group, prefix)
        each = q.transpose(0, 1).reshape(batch * kv, n_q * group, dim)
        k, w = (tokens(s[p], table[1:], suffix).view(batch * kv, suffix, dim) for p in ("k_pool", "v_pool"))
        b = (torch.bmm(each, k.transpose(1, 2).contiguous()) * s["scale"]).view(batch, kv, n_q, group, suffix)
        limit = held[:, None] - n_q + 1 + torch.arange(n_q, device=DEV)  # tokens each query sees, its own the last
        seen = torch.arange(suffix, device=DEV) < limit[:, None, :, None, None]
        b = b.masked_fill(~seen, -math.inf).view(batch, kv, n_q * group, suffix).transpose(0, 1)
        top = b.amax(-1, keepdim=True)
        if prefix:
            top = torch.maximum(top, a.amax(-1, keepdim=True))
        at = torch.where(top == -math.inf, 0.0, top)
        a, b = (a - at).exp(), (b - at).exp()
        total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
        o = torch.bmm(a.reshape(kv, batch * n_q * group, prefix), v).view(kv, batch, n_q * group, dim)
        o = o + torch.bmm(b.transpose(0, 1).reshape(batch * kv, n_q * group, suffix), w).view(
            batch, kv, n_q * group, dim).transpose(0, 1)
        o = torch.where(total > 0, o / total, 0.0)
        lse = at + total.log()

        def back(x):
            return x.view(kv, batch, n_q, group, -1).permute(1, 2, 0, 3, 4).reshape(batch, n_q, kv * group, -1)

        return back(o).to(s["q"].dtype), back(lse)[..., 0].contiguous()


def run(state):
    c = state["case"]
    if own:
        return getattr(_Own, c["op"])(c, state, torch.cuda.current_stream().cuda_stream)
    return getattr(_Plain, c["op"])(c, state)


# ---- what a pass cannot do without -----------------------------------------

_SIZES = {"f16": 2, "bf16": 2, "f32": 4}


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 2 * n * _SIZES[c["dtype"]] + 4 * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        n = c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * n * _SIZES[c["dtype"]] + 12 * c["tokens"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot"]}
    page = 2 * c["slots"] * c["heads"] * c["dim"] if "pools" in c else 0
    if c["op"] == "fork":  # half of a row's pages on average, read and written in the table and counted
        entries = c["children"] * (c["row_tokens"] / 2 / c["slots"] + 1)
        copies = c["children"] * (1 - 1 / c["slots"])
        return {"bytes": 2 * page * c["pools"] * copies + 16 * entries + 4 * c["pages"], "flops": 0}
    if c["op"] == "compact":
        row_pages = -(-c["row_tokens"] // c["slots"])
        share = min(c["used"], c["rows"] * row_pages / c["pages"])
        return {"bytes": 2 * page * c["pools"] * c["pages"] * share * (1 - share) + 8 * c["pages"]
                + 8 * c["rows"] * row_pages, "flops": 0}
    tokens = c["prefix"] + c["batch"] * c["suffix"] / 2
    q = c["batch"] * c["q_len"] * c["heads"]
    return {"bytes": 2 * (2 * tokens * c["kv_heads"] * c["dim"] + 2 * q * c["dim"]) + 4 * q,
            "flops": 4 * q * c["dim"] * (c["prefix"] + c["suffix"] / 2)}


# ---- the definitions in 64 bits --------------------------------------------

def _turned(x, pos, c):
    """Each pair of x as a complex number times magnitude * exp(i * pos * frequency), in 64 bits."""
    n, d = c["rot"], x.shape[-1]
    scaling, factor = c.get("scaling", "none"), c.get("factor", 1.0)
    theta = []
    for j in range(n // 2):
        b = 10000.0 * (factor ** (n / (n - 2)) if scaling == "base" and n > 2 else 1.0)
        f = math.exp(-2.0 * j / n * math.log(b))
        if scaling == "linear":
            f /= factor
        elif scaling == "ramp":
            share = (4096 * f / (2 * math.pi) - 1.0) / 31.0
            share = min(1.0, max(0.0, share))
            f = share * f + (1.0 - share) * f / factor
        theta.append(f)
    turn = pos.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=x.device)
    if c.get("inverse"):
        turn = -turn
    turn = torch.polar(torch.full_like(turn, c.get("magnitude", 1.0)), turn)[:, None]
    y = x.double().clone()
    first, second = (slice(0, n, 2), slice(1, n, 2)) if c["layout"] == "interleaved" else (slice(0, n // 2),
                                                                                         slice(n // 2, n))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers alone
    s = {"case": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    getattr(_Inputs, case["op"])(case, g, np.random.default_rng(seed), s)
    c = case
    if c["op"] == "rope":
        return _turned(s["x"], s["pos"], c)
    if c["op"] == "append":
        k = _turned(s["k"], s["pos"], c)
        pools = [s["k_pool"].double(), s["v_pool"].double()]
        page_of = s["table"][s["rows"].long(), s["at"].long().div(c["slots"], rounding_mode="floor")].long()
        for pool, new in zip(pools, (k, s["v"].double())):
            view = pool.transpose(1, 2) if c["heads_first"] else pool
            view[page_of, s["at"].long().remainder(c["slots"])] = new
        return _turned(s["q"], s["pos"], c), pools[0], pools[1]
    # attention, one sequence and one shared head after the other
    batch, n_q, kv, slots = c["batch"], c["q_len"], c["kv_heads"], c["slots"]
    group = c["heads"] // kv
    k_pool, v_pool = ((s[n].transpose(1, 2) if c["heads_first"] else s[n]) for n in ("k_pool", "v_pool"))
    table, held = s["table"].cpu().tolist(), s["lens"].cpu().tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)

    def of_row(pool, row, count):
        pages = torch.tensor(table[row][:-(-count // slots)], dtype=torch.long, device=DEV)
        return pool[pages].flatten(0, 1)[:count].double().transpose(0, 1).contiguous()  # [kv, count, dim]

    head_k, head_v = of_row(k_pool, 0, held[0]), of_row(v_pool, 0, held[0])
    for b in range(batch):
        k = torch.cat((head_k, of_row(k_pool, b + 1, held[b + 1])), 1)
        v = torch.cat((head_v, of_row(v_pool, b + 1, held[b + 1])), 1)
        for j in range(n_q):
            sees = c["prefix"] + max(0, held[b + 1] - (n_q - 1 - j))
            if sees == 0:
                continue
            q = s["q"][b, j].double().view(kv, group, c["dim"])
            score = torch.matmul(q, k[:, :sees].transpose(1, 2).contiguous()) * s["scale"]
            out[b, j] = torch.matmul(torch.softmax(score, -1), v[:, :sees].contiguous()).flatten(0, 1)
            lse[b, j] = torch.logsumexp(score, -1).flatten()
    return out, lse
