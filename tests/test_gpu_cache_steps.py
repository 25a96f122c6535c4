"""The cache's calls together, as a program would make them: prompts in chunks,
single tokens behind a window, drafted trees of which some tokens are kept, rows
forked and given back, on pools of 16 bits and of codes.  Every step's result is
compared with dense attention in 64 bits over the tokens that the test's own
record says each row holds."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_attn_cache import parents_of  # noqa: E402
from test_gpu_kvcache import TORCH, f64, gen, ints, tensor_map  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


class Cache:
    def __init__(self, dtype, fmt, rows, row_tokens, slots, heads, kv, dim, window, sinks, g):
        self.dtype, self.fmt, self.slots, self.heads, self.kv, self.dim = dtype, fmt, slots, heads, kv, dim
        self.window, self.sinks, self.g = window, sinks, g
        row_pages = -(-row_tokens // slots)
        self.pages = rows * row_pages
        each = slots if fmt == "same" else ok.code_rows(slots, dim)
        kind = TORCH[dtype] if fmt == "same" else torch.uint8
        self.pools = [torch.zeros((self.pages, each, kv, dim), dtype=kind, device="cuda") for _ in "kv"]
        name = dtype if fmt == "same" else "u8"
        self.maps = [tensor_map(p.transpose(1, 2), name) for p in self.pools]
        self.all_maps = att.tmap_array(self.maps)
        self.table = torch.full((rows, row_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(self.pages, dtype=torch.int32, device="cuda")
        self.pt = att.page_table(self.table, self.lens, self.refs, self.pages, slots)
        self.ws = torch.empty(att.page_workspace(self.pt, rows), dtype=torch.uint8, device="cuda")
        self.plan = att.rope_encode(dim, "half", 10000.0)
        self.thetas = ok.rope_thetas(dim)
        self.record = [[] for _ in range(rows)]                          # each row's tokens: (key, value) before the cache

    def append(self, rows, pos, q, k, v):
        """[len(rows), n, ...]: the tokens of each row at its end; positions [len(rows), n].  Returns the turned queries."""
        b, n = q.shape[:2]
        good = ints([0] * b)
        start = self.lens[ints(rows).long()].clone()
        att.page_extend(self.pt, ints(rows), ints([n] * b), b, good, self.ws, stream())
        assert good.tolist() == [1] * b
        flat = [t.reshape(b * n, t.shape[2], self.dim) for t in (q, k, v)]
        out = torch.empty_like(flat[0])
        d_rows = ints(np.repeat(rows, n))
        d_at = (start[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)).reshape(-1).int().contiguous()
        maps = [tensor_map(t, self.dtype) for t in (flat[0], out, flat[1], flat[2])]
        args = (*self.maps, self.pt, d_rows, d_at, ints(pos.reshape(-1)), stream())
        if self.fmt == "same":
            att.rope_append(self.plan, *maps, *args)
        else:
            att.kv8_append(self.plan, *maps, self.fmt, *args)
        turned = ok.rope(f64(flat[1]), pos.reshape(-1), self.thetas)[0].reshape(b, n, self.kv, self.dim)
        for i, r in enumerate(rows):
            self.record[r] += [(turned[i, j], f64(v)[i, j]) for j in range(n)]
        return out.view(q.shape)

    def attend(self, rows, q, parents=None, hint=None):
        b, n = q.shape[:2]
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        mq, mo = tensor_map(q, self.dtype), tensor_map(o, self.dtype)
        hint = int(self.lens.max()) if hint is None else hint
        ws = torch.empty(att.attn_cache_workspace(mq, self.maps[0], self.window, self.sinks, hint), dtype=torch.uint8,
                         device="cuda")
        scale = 1 / math.sqrt(self.dim)
        args = (self.window, self.sinks, hint, scale, mo, lse, ws, stream())
        if parents is None:
            att.attn_window(mq, *self.maps, self.fmt, self.pt, ints(rows), None, *args)
        else:
            att.attn_tree(mq, *self.maps, self.fmt, self.pt, ints(rows), None, ints(parents), *args)
        self.check(rows, q, o, lse, parents)
        return o

    def check(self, rows, q, o, lse, parents):
        """Codes are off by half a step, 1/254 of the largest element of a head (int8) or 2^-4 of each element (e4m3),
        and a scale by 2^-7 at most; 16 bits by half a step.  A key's error e shifts a score by scale * |q| . e, which
        shifts the result by twice that of the largest value's size; a value's own error is at most what it is."""
        step = ok.half_step(self.dtype)
        for i, r in enumerate(rows):
            k, v = (np.stack([t[x] for t in self.record[r]]) for x in (0, 1))
            sees = ok.causal_sees(len(k), q.shape[1], self.window, self.sinks) if parents is None else \
                ok.tree_sees(len(k), [int(p) for p in parents[i]], self.window, self.sinks)
            scale = 1 / math.sqrt(self.dim)
            want, want_lse, weight, size, n = ok.attend(f64(q)[i], k, v, sees, scale)
            if self.fmt == "int8":
                # absolute: half a code of the head's largest element
                ek = np.abs(k).max(-1, keepdims=True) * (1 + 2.0 ** -7) / 254 + 0 * k
                ev = np.abs(v).max() * (1 + 2.0 ** -7) / 254
            elif self.fmt == "e4m3":
                ek, ev = np.abs(k) * 2.0 ** -4 + np.abs(k).max(-1, keepdims=True) * 2.0 ** -18, np.abs(v).max() * 2.0 ** -4
            else:
                ek, ev = np.abs(k) * step, 0.0
            shift = np.zeros(lse.shape[1:])
            group = self.heads // self.kv
            for h in range(self.heads):
                e = scale * np.abs(f64(q)[i, :, h]) @ ek[:, h // group].T
                shift[:, h] = np.where(sees, e, 0).max(1)
            shift += 2.0 ** -20 * size + 2.0 ** -20                      # the rotation's and the products' roundings
            # weights change by a factor of exp(shift) up or down, and so does their sum
            limit = np.expm1(2 * shift)[..., None] * (weight + np.abs(want)) + ev * np.exp(2 * shift)[..., None]
            limit += 4 * step * (weight + np.abs(want)) + 1e-6
            assert (np.abs(f64(o)[i] - want) <= limit).all()
            assert (np.abs(f64(lse)[i] - want_lse) <= shift + 2.0 ** -19 * np.abs(want_lse)).all()


@pytest.mark.parametrize("dtype,fmt,window,sinks", [("bf16", "same", 0, 0), ("f16", "int8", 40, 3), ("bf16", "e4m3", 25, 2),
                                                    ("f16", "same", 17, 4), ("bf16", "int8", 0, 0)])
def test_serving(dtype, fmt, window, sinks):
    g = gen(900)
    rng = np.random.default_rng(3)
    c = Cache(dtype, fmt, 6, 200, 8, 4, 2, 64, window, sinks, g)

    def tokens(b, n):
        return [torch.randn((b, n, h, c.dim), generator=g).to(TORCH[dtype]).cuda() for h in (c.heads, c.kv, c.kv)]

    def causal(rows, n, hint=None):
        start = np.array([len(c.record[r]) for r in rows])
        q = c.append(rows, start[:, None] + np.arange(n), *tokens(len(rows), n))
        c.attend(rows, q, hint=hint)

    def drafted(rows, n, most):
        parents = parents_of(g, len(rows), n, "near")
        depth = np.zeros((len(rows), n), int)
        for i in range(len(rows)):
            for j in range(n):
                depth[i, j] = 0 if parents[i, j] < 0 else depth[i, parents[i, j]] + 1
        base = np.array([len(c.record[r]) for r in rows])
        q = c.append(rows, base[:, None] + depth, *tokens(len(rows), n))
        c.attend(rows, q, parents)
        # accept a way down the tree, not longer than `most`
        keep, count = np.full((len(rows), most), -1), np.zeros(len(rows), int)
        for i in range(len(rows)):
            way = [int(rng.integers(0, n))]
            while parents[i, way[-1]] >= 0:
                way.append(int(parents[i, way[-1]]))
            way = way[::-1][:most]
            keep[i, :len(way)], count[i] = way, len(way)
        good = ints([0] * len(rows))
        att.page_keep(c.pt, c.all_maps, ints(rows), ints(base), ints(keep), ints(count), len(rows), good, stream())
        assert good.tolist() == [1] * len(rows)
        for i, r in enumerate(rows):
            c.record[r] = c.record[r][:base[i]] + [c.record[r][base[i] + k] for k in keep[i, :count[i]]]
        assert c.lens.tolist() == [len(t) for t in c.record]

    causal([0, 2, 4], 50)                                                # prompts, in two chunks
    causal([0, 2, 4], 13, hint=1 << 20)
    for _ in range(3):
        causal([0, 2, 4], 1)
        drafted([4, 0, 2], 11, 5)
    good = ints([0, 0])
    att.page_fork(c.pt, c.all_maps, ints([2, 0]), ints([1, 5]), 2, good, c.ws, stream())
    assert good.tolist() == [1, 1]
    c.record[1], c.record[5] = list(c.record[2]), list(c.record[0])
    drafted([1, 2, 5, 0], 9, 4)                                          # twins go on by themselves
    causal([1, 2, 5, 0], 2)
    att.page_free(c.pt, ints([2, 4]), 2, stream())
    c.record[2], c.record[4] = [], []
    used = ints([0])
    att.page_compact(c.pt, c.pt, c.all_maps, used, c.ws, stream())
    assert used.item() == int((c.refs > 0).sum())
    causal([5, 1, 0], 1)
    causal([3, 2], 30)
    drafted([5, 3], 40, 8)
    causal([0, 1, 2, 3, 5], 1)
    if fmt != "same":                                                    # a row taken out of the cache
        n = len(c.record[5])
        k, v = (torch.empty((n, c.kv, c.dim), dtype=TORCH[dtype], device="cuda") for _ in "kv")
        att.kv8_read(fmt, *c.maps, c.pt, ints([5] * n), ints(np.arange(n)), tensor_map(k, dtype), tensor_map(v, dtype),
                     stream())
        want = np.stack([t[1] for t in c.record[5]])
        top = np.abs(want).max(-1, keepdims=True)
        half = top * (1 + 2.0 ** -7) / 254 if fmt == "int8" else np.abs(want) * 2.0 ** -4 + top * 2.0 ** -18
        assert (np.abs(f64(v) - want) <= half + 2 * ok.half_step(dtype) * top).all()
    att.tile_device_status(stream())


def test_a_captured_step():
    """One decode step of an 8-bit cache, captured once: extend, append, attend.  Lengths, tables and positions follow."""
    g = gen(901)
    dtype, fmt, n = "bf16", "int8", 3
    c = Cache(dtype, fmt, n, 300, 16, 4, 2, 64, 64, 4, g)
    rows = list(range(n))
    start = [70, 15, 200]
    for r, t in zip(rows, start):
        q, k, v = (torch.randn((1, t, h, c.dim), generator=g).to(TORCH[dtype]).cuda() for h in (4, 2, 2))
        c.append([r], np.arange(t)[None], q, k, v)
    q, k, v = (torch.zeros((n, 1, h, c.dim), dtype=TORCH[dtype], device="cuda") for h in (4, 2, 2))
    flat = [t.view(n, t.shape[2], c.dim) for t in (q, k, v)]
    turned, o = torch.zeros_like(flat[0]), torch.zeros_like(q)
    lse = torch.zeros(q.shape[:3], device="cuda")
    d_rows, one, good, at = ints(rows), ints([1] * n), ints([0] * n), ints([0] * n)
    maps = [tensor_map(t, dtype) for t in (flat[0], turned, flat[1], flat[2])]
    mq, mo = tensor_map(turned.view(q.shape), dtype), tensor_map(o, dtype)
    ws = torch.empty(att.attn_cache_workspace(mq, c.maps[0], 64, 4, 300), dtype=torch.uint8, device="cuda")

    def step(st):
        at.copy_(c.lens)
        att.page_extend(c.pt, d_rows, one, n, good, c.ws, st)
        att.kv8_append(c.plan, *maps, fmt, *c.maps, c.pt, d_rows, at, at, st)
        att.attn_window(mq, *c.maps, fmt, c.pt, d_rows, None, 64, 4, 300, 0.125, mo, lse, ws, st)

    state = [c.table, c.lens, c.refs, *c.pools]
    saved = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(torch.cuda.current_stream().cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for t, old in zip(state, saved):
        t.copy_(old)
    for i in range(20):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        pos = np.array([[len(c.record[r])] for r in rows])
        graph.replay()
        torch.cuda.synchronize()
        new = ok.rope(f64(flat[1]), pos[:, 0], c.thetas)[0]
        for r in rows:
            c.record[r].append((new[r], f64(v)[r, 0]))
        assert good.tolist() == [1] * n
        c.check(rows, turned.view(q.shape), o, lse, None)
