"""Parallel sampling over a paged cache: one prompt, several answers, two layers.

The prompt's keys and values are written once (row 0 of the page table); the
answers' rows hold their own tokens alone and attend to the prompt as a shared
prefix.  Every few steps the worse half of the answers is given up and the
better half is forked (full pages shared, the unfinished page copied); at the
end the pages that are left move together.  A decode step is captured into a
graph once and replayed: lengths, tables and positions live on the device.

    python examples/paged_decode.py [--steps 24] [--answers 8] [--prompt 300]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import async_tensor_tile_amd as att  # noqa: E402

NAMES = {torch.bfloat16: "bf16", torch.float16: "f16"}


def tensor_map(t: torch.Tensor) -> att.tmap_t:
    """The tensor map of a torch tensor, dimensions innermost first."""
    e = t.element_size()
    return att.tmap_encode(NAMES[t.dtype], t.dim(), t.data_ptr(), tuple(reversed(t.shape)),
                           tuple(s * e for s in reversed(t.stride()[:-1])), (16 // e,) + (1,) * (t.dim() - 1))


class Cache:
    """Page table and pools of a model: `layers` pairs of pools
    [pages, slots, kv heads, dim], rows of at most `row_tokens` tokens."""

    def __init__(self, layers, pages, slots, kv, dim, rows, row_tokens, dtype=torch.bfloat16):
        new = dict(device="cuda")
        self.pages, self.slots, self.rows = pages, slots, rows
        self.table = torch.full((rows, -(-row_tokens // slots)), -1, dtype=torch.int32, **new)
        self.lens = torch.zeros(rows, dtype=torch.int32, **new)
        self.refs = torch.zeros(pages, dtype=torch.int32, **new)
        self.pools = [tuple(torch.zeros((pages, slots, kv, dim), dtype=dtype, **new) for _ in "kv") for _ in range(layers)]
        self.maps = [tuple(tensor_map(p.transpose(1, 2)) for p in pair) for pair in self.pools]
        self.all_maps = att.tmap_array([m for pair in self.maps for m in pair])
        self.pt = att.page_table(self.table, self.lens, self.refs, pages, slots)
        self.ws = torch.empty(att.page_workspace(self.pt, rows), dtype=torch.uint8, **new)
        self.ok = torch.ones(rows, dtype=torch.int32, **new)

    def extend(self, rows, add):
        att.page_extend(self.pt, rows, add, rows.numel(), self.ok, self.ws, stream())

    def fork(self, src, dst):
        att.page_fork(self.pt, self.all_maps, src, dst, src.numel(), self.ok, self.ws, stream())

    def free(self, rows):
        att.page_free(self.pt, rows, rows.numel(), stream())

    def compact(self):
        used = torch.zeros(1, dtype=torch.int32, device="cuda")
        att.page_compact(self.pt, self.pt, self.all_maps, used, self.ws, stream())
        return used


def stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def ints(v) -> torch.Tensor:
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """Embedding, `layers` of attention with a residual, logits; random weights."""

    def __init__(self, layers=2, vocab=512, heads=8, kv=2, dim=64, seed=0, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.layers, self.heads, self.kv, self.dim, width = layers, heads, kv, dim, heads * dim

        def weights(*shape):
            return (torch.randn(shape, generator=g) / shape[0] ** 0.5).to(dtype).cuda()

        self.embed = (torch.randn((vocab, width), generator=g) / 2).to(dtype).cuda()
        self.wq = [weights(width, width) for _ in range(layers)]
        self.wk = [weights(width, kv * dim) for _ in range(layers)]
        self.wv = [weights(width, kv * dim) for _ in range(layers)]
        self.wo = [weights(width, width) for _ in range(layers)]
        self.head = weights(width, vocab)
        self.plan = att.rope_encode(dim, "half", 10000.0, "ramp", 4.0, 4096)


class Runner:
    """The buffers, maps and workspace of one shape of call: `batch` rows of
    `q_len` new tokens behind a prefix of prefix_len tokens in row 0."""

    def __init__(self, model, cache, rows, q_len, prefix_len, hint):
        m, n, dt = model, rows.numel() * q_len, model.embed.dtype
        self.m, self.cache, self.rows, self.q_len, self.prefix, self.hint = m, cache, rows, q_len, prefix_len, hint
        new = dict(device="cuda", dtype=dt)
        self.q, self.turned, self.o = (torch.empty((n, m.heads, m.dim), **new) for _ in range(3))
        self.k, self.v = (torch.empty((n, m.kv, m.dim), **new) for _ in range(2))
        shape = (rows.numel(), q_len, m.heads, m.dim)
        self.mq, self.mo = tensor_map(self.turned.view(shape)), tensor_map(self.o.view(shape))
        self.maps = [tensor_map(t) for t in (self.q, self.turned, self.k, self.v)]
        self.ws = torch.empty(att.attn_workspace(self.mq, cache.maps[0][0], prefix_len, hint), dtype=torch.uint8,
                              device="cuda")
        self.token_rows = rows.repeat_interleave(q_len)
        self.offset = torch.arange(q_len, dtype=torch.int32, device="cuda").repeat(rows.numel())
        self.add = torch.full_like(rows, q_len)

    def __call__(self, tokens):
        """Logits of `tokens` [batch * q_len], appended to their rows."""
        m, c = self.m, self.cache
        at = c.lens[self.token_rows.long()] + self.offset
        pos = at + self.prefix
        c.extend(self.rows, self.add)
        x = m.embed[tokens]
        for layer in range(m.layers):
            self.q.view(x.shape[0], -1).copy_(x @ m.wq[layer])
            self.k.view(x.shape[0], -1).copy_(x @ m.wk[layer])
            self.v.view(x.shape[0], -1).copy_(x @ m.wv[layer])
            mk, mv = c.maps[layer]
            att.rope_append(m.plan, *self.maps, mk, mv, c.pt, self.token_rows, at, pos, stream())
            att.attn_shared_prefix(self.mq, mk, mv, c.pt, 0, self.prefix, self.rows, self.hint, m.dim ** -0.5, self.mo,
                                   None, self.ws, stream())
            x = x + self.o.view(x.shape[0], -1) @ m.wo[layer]
        return x.float() @ m.head.float()


def generate(steps=24, answers=8, prompt=300, every=8, slots=16, seed=0):
    """The answers' tokens [answers, steps], the model, the prompt's tokens and
    the cache (every row but the prompt's an answer)."""
    model = Model(seed=seed)
    per = -(-steps // slots) + 1
    cache = Cache(model.layers, -(-prompt // slots) + 2 * answers * per, slots, model.kv, model.dim, 1 + 2 * answers,
                  max(prompt, steps))
    g = torch.Generator().manual_seed(seed + 1)
    prompt_tokens = torch.randint(0, model.embed.shape[0], (prompt,), generator=g).cuda()
    last = Runner(model, cache, ints([0]), prompt, 0, prompt)(prompt_tokens)[-1]

    top = last.topk(answers)
    token, score = top.indices.clone(), top.values.log_softmax(0)         # the answers' first tokens
    history = token[:, None].clone()
    rows = ints(range(1, answers + 1))
    step = Runner(model, cache, rows, 1, prompt, steps)                  # reads `rows` on the device

    def decode():
        p = step(token).log_softmax(-1).max(-1)
        token.copy_(p.indices)
        score.add_(p.values)

    state = [cache.table, cache.lens, cache.refs, token, score]
    saved = [s.clone() for s in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()                                                         # warm-up: undone below
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            decode()
    torch.cuda.current_stream().wait_stream(side)
    for s, old in zip(state, saved):
        s.copy_(old)

    for i in range(1, steps):
        graph.replay()
        history = torch.cat((history, token[:, None]), 1)
        if i % every == 0:                                               # the better half goes on twice
            order = score.argsort(descending=True)
            keep, drop = order[:answers - answers // 2], order[answers - answers // 2:]
            twin = keep[:drop.numel()]
            cache.free(rows[drop].contiguous())
            cache.fork(rows[twin].contiguous(), rows[drop].contiguous())
            token[drop], score[drop], history[drop] = token[twin], score[twin] - 1e-3, history[twin]
    used = cache.compact()
    att.tile_device_status(stream())
    assert used.item() == int((cache.refs > 0).sum())
    return history, model, prompt_tokens, cache


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--answers", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    args = ap.parse_args()
    generate(args.steps, args.answers, args.prompt)
    torch.cuda.synchronize()
    t = time.perf_counter()
    history, _, _, cache = generate(args.steps, args.answers, args.prompt)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) * 1e3
    print(f"{args.answers} answers of {args.steps} tokens behind {args.prompt}: {ms:.1f} ms, "
          f"{int((cache.refs > 0).sum())} of {cache.pages} pages in use")
    print(history[:, :8].tolist())


if __name__ == "__main__":
    main()
