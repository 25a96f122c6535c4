"""GPU parity of the attention over the cache, with a window or of a tree,
against the 64-bit oracle.

Tolerances count roundings.  One rounding to a type is off by at most half a
step (bf16 2^-8, fp16 2^-11, fp32 2^-24, relative).  A score is a sum of dim
products in fp32 (codes and keys of 16 bits are exact in them), times a key's
scale and the call's: off by at most (dim + 8) * 2^-24 times the sum of their
absolute values, which shifts a weight by as much again, relatively, and the
exponential adds 2^-21.  Each weight, times its value's scale or a part of it, is
rounded to the type for the product with the values or their codes; n of those
are added in fp32, and the quotient is rounded to the type.  Weights and values
below the smallest normal number of f16 are off by at most 2^-25."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_kvcache import TORCH, f64, gen, ints, padded, tensor_map  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


class Setup:
    """Sequences of given lengths over pools whose pages lie in any order, with
    rows that the batch does not use and pages that no row holds."""

    def __init__(self, g, dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, heads_first=False, gap=0, spare=2,
                 junk=float("nan")):
        self.dtype, self.fmt, self.slots, self.kv, self.heads_first = dtype, fmt, slots, kv, heads_first
        self.seq_lens, self.counts, self.q_len, self.dim = lens, counts, q_len, dim
        batch = len(lens)
        each = [-(-n // slots) for n in lens]
        pages = sum(each) + spare
        self.pages = pages
        order, at = torch.randperm(pages, generator=g).tolist(), 0
        self.rows = torch.randperm(batch + 2, generator=g)[:batch].tolist()
        table = np.full((batch + 2, max(each + [1])), -1, np.int32)
        length = np.zeros(batch + 2, np.int32)
        for b, r in enumerate(self.rows):
            table[r, :each[b]] = order[at:at + each[b]]
            length[r] = lens[b]
            at += each[b]
        self.table, self.lens, self.d_rows = ints(table), ints(length), ints(self.rows)
        self.count = None if counts is None else ints(counts)
        self.k, self.v = (self.pool(g, pages, gap) for _ in "kv")
        self.pt = att.page_table(self.table, self.lens, None, pages, slots)
        _, self.q = padded((batch, q_len, heads, dim), dtype, gap, g)
        whole = torch.full((batch, q_len, heads, dim + gap + (16 if gap else 0)), -3.0, dtype=TORCH[dtype]).cuda()
        self.o_whole, self.o = whole, whole[..., :dim]
        self.lse = torch.full(self.q.shape[:3], -3.0, device="cuda")

    def pool(self, g, pages, gap):
        n, kv, dim = self.slots, self.kv, self.dim
        if self.fmt == "same":
            shape = (pages, kv, n, dim) if self.heads_first else (pages, n, kv, dim)
            return padded(shape, self.dtype, gap, g)[1]
        rows = ok.code_rows(n, dim)
        p = torch.zeros((pages, kv, rows, dim + 16 * (gap > 0)), dtype=torch.uint8)
        top = 127 if self.fmt == "int8" else 126                          # every number but NaN
        code = torch.randint(-top, top + 1, (pages, kv, n, dim), generator=g)
        code = code.to(torch.int8).view(torch.uint8) if self.fmt == "int8" else \
            (code.abs() + 128 * (code < 0)).to(torch.uint8)
        if self.fmt == "e4m3":                                            # of the sizes that a scaled head has
            code = torch.where(code & 127 > 0x60, code & 0xE7, code)
        p[:, :, :n, :dim] = code
        unit = 1 / 60 if self.fmt == "int8" else 1 / 16
        scale = (unit * torch.exp(0.5 * torch.randn((pages, kv, n), generator=g))).bfloat16()
        tail = torch.zeros((pages, kv, (rows - n) * dim), dtype=torch.uint8)
        tail[..., :2 * n] = scale.view(torch.uint8)
        p[:, :, n:, :dim] = tail.view(pages, kv, rows - n, dim)
        return (p if self.heads_first else p.transpose(1, 2).contiguous()).cuda()[..., :dim]

    def map(self, p):
        return tensor_map(p if self.heads_first else p.transpose(1, 2), self.dtype if self.fmt == "same" else "u8")

    def tokens(self, p, b):
        """[length, kv, dim] of sequence b, in 64 bits."""
        n = self.seq_lens[b]
        t = self.table[self.rows[b], :-(-n // self.slots)].long()
        x = p[t] if self.heads_first else p[t].transpose(1, 2)            # [pages, kv, rows, dim]
        if self.fmt == "same":
            x = f64(x)
        else:
            code, scale = ok.split_codes(x.cpu().numpy(), self.slots, self.fmt)
            x = code * scale[..., None]
        return x.swapaxes(1, 2).reshape(-1, self.kv, self.dim)[:n]

    def run(self, window=0, sinks=0, parents=None, scale=None, hint=None, ws=None, rows=True, lse=True, st=None):
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        hint = max(self.seq_lens) if hint is None else hint
        mq, mk, mv, mo = tensor_map(self.q, self.dtype), self.map(self.k), self.map(self.v), tensor_map(self.o, self.dtype)
        if ws is None:
            size = att.attn_cache_workspace(mq, mk, window, sinks, hint)
            assert size > 0
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        st = stream() if st is None else st
        d_rows, l = self.d_rows if rows else None, self.lse if lse else None
        if parents is None:
            att.attn_window(mq, mk, mv, self.fmt, self.pt, d_rows, self.count, window, sinks, hint, scale, mo, l, ws, st)
        else:
            att.attn_tree(mq, mk, mv, self.fmt, self.pt, d_rows, self.count, parents, window, sinks, hint, scale, mo, l,
                          ws, st)
        return f64(self.o), f64(self.lse)

    def check(self, window=0, sinks=0, parents=None, scale=None, **kw):
        d_parents = None if parents is None else ints(parents)
        got, got_lse = self.run(window, sinks, d_parents, scale, **kw)
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        q, step = f64(self.q), ok.half_step(self.dtype)
        for b, length in enumerate(self.seq_lens):
            n = self.q_len if self.counts is None else self.counts[b]
            assert (got[b, n:] == -3.0).all() and (got_lse[b, n:] == -3.0).all()
            if n == 0:
                continue
            k, v = self.tokens(self.k, b), self.tokens(self.v, b)
            sees = ok.causal_sees(length, n, window, sinks) if parents is None else \
                ok.tree_sees(length, [int(p) for p in parents[b][:n]], window, sinks)
            want, lse, weight, size, seen = ok.attend(q[b, :n], k, v, sees, scale)
            shift = (self.dim + 8) * 2.0 ** -24 * size + 2.0 ** -21
            m = seen[..., None]
            limit = weight * (step + 2 * shift[..., None] + (m + 32) * 2.0 ** -24)
            tiny = 2.0 ** -25 if self.dtype == "f16" else 1e-37
            limit += step * np.abs(want) + (m + 1) * tiny * (8 if self.fmt == "same" else 16)
            off = np.abs(got[b, :n] - want)
            assert (off <= limit).all(), (b, (off - limit).max(), np.argwhere(off > limit)[:4])
            empty = np.isneginf(lse)
            assert np.array_equal(np.isneginf(got_lse[b, :n]), empty) and (got[b, :n][empty] == 0).all()
            with np.errstate(invalid="ignore"):
                off = np.abs(got_lse[b, :n] - lse)
            near = shift + (seen + 32) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, lse))
            assert (off <= near)[~empty].all(), (b, off[~empty].max())
        assert (self.o_whole[..., self.dim:] == -3.0).all()
        return got, got_lse


# dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, heads_first, gap, window, sinks, hint
WINDOW = [
    ("f16", "same", [1], None, 1, 1, 1, 8, 1, False, 0, 0, 0, 0),
    ("bf16", "same", [5, 0, 40, 33], None, 1, 8, 2, 64, 16, False, 0, 0, 0, None),
    ("f16", "same", [700, 129, 3], None, 1, 8, 2, 64, 16, False, 0, 128, 4, None),
    ("bf16", "same", [700, 1500, 2, 513], [1, 3, 2, 0], 3, 32, 8, 128, 48, True, 8, 100, 7, 4000),
    ("f16", "same", [300, 299], None, 5, 10, 2, 80, 7, False, 16, 1, 0, None),
    ("bf16", "same", [2000], None, 2, 6, 3, 96, 100, False, 0, 33, 5, 5000),
    ("f16", "same", [400, 90], [4, 1], 4, 4, 4, 160, 8, True, 0, 70, 70, 2000),
    ("bf16", "same", [260, 31], None, 3, 2, 1, 256, 64, False, 8, 200, 1, None),
    ("bf16", "int8", [5, 0, 40, 700], None, 1, 8, 2, 64, 16, False, 0, 0, 0, None),
    ("f16", "e4m3", [700, 129, 3], [1, 1, 1], 2, 8, 2, 128, 16, True, 16, 128, 4, 3000),
    ("f16", "int8", [1100, 64], None, 3, 10, 2, 80, 48, False, 16, 50, 3, 3000),
    ("bf16", "e4m3", [400, 33], None, 2, 4, 2, 96, 5, True, 0, 1, 1, None),
    ("f16", "int8", [300, 7], None, 1, 3, 1, 192, 100, False, 0, 90, 2, None),
    ("bf16", "e4m3", [513, 1], None, 4, 2, 2, 240, 16, False, 0, 0, 0, 2000),
    # many rows
    ("bf16", "same", [200], None, 200, 4, 1, 64, 16, False, 0, 0, 0, None),
    ("f16", "same", [300, 70, 5], [150, 70, 20], 150, 8, 2, 128, 16, False, 8, 40, 4, 0),
    ("bf16", "same", [1500, 600], [257, 300], 300, 2, 2, 128, 48, True, 0, 500, 3, None),
    ("bf16", "same", [1000], None, 65, 3, 3, 96, 33, False, 0, 64, 0, 4000),
    ("f16", "same", [700], None, 64, 6, 2, 72, 16, True, 0, 0, 0, 20000),
    ("bf16", "same", [513, 100], [70, 100], 100, 4, 2, 192, 16, False, 0, 77, 5, None),
    ("f16", "same", [450], None, 129, 2, 1, 256, 8, False, 0, 130, 2, None),
    ("bf16", "int8", [777, 200], [300, 133], 300, 5, 1, 80, 48, True, 0, 300, 3, None),
    ("f16", "e4m3", [1300], None, 100, 8, 2, 128, 16, False, 16, 0, 0, 5000),
    ("f16", "int8", [900, 66], [80, 66], 80, 4, 4, 64, 16, False, 0, 100, 1, None),
    ("bf16", "e4m3", [600], None, 90, 2, 1, 192, 16, True, 0, 55, 55, None),
    ("f16", "e4m3", [333], None, 140, 1, 1, 96, 1, False, 0, 0, 0, None),
    ("bf16", "int8", [600, 0, 3], [128, 5, 128], 128, 2, 1, 256, 16, False, 0, 0, 0, 3000),
    ("bf16", "same", [40, 0, 100], None, 100, 4, 2, 64, 16, False, 0, 30, 4, None),   # more queries than tokens
]


@pytest.mark.parametrize("case", range(len(WINDOW)))
def test_window(case):
    dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first, gap, window, sinks, hint = WINDOW[case]
    s = Setup(gen(400 + case), dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first, gap)
    s.check(window, sinks, hint=hint)


def parents_of(g, batch, n, kind):
    if kind == "chain":
        return np.tile(np.arange(n) - 1, (batch, 1))
    if kind == "star":
        return np.full((batch, n), -1)
    back = torch.randint(1, {"near": 4, "far": n + 2}[kind], (batch, n), generator=g).numpy()
    return np.maximum(np.arange(n)[None] - back, -1)


# dtype, fmt, lens, counts, nodes, heads, kv, dim, slots, heads_first, gap, window, sinks, hint, kind
TREE = [
    ("f16", "same", [1], None, 1, 1, 1, 8, 1, False, 0, 0, 0, 0, "star"),
    ("bf16", "same", [30, 13, 200], [13, 13, 5], 13, 2, 1, 64, 16, False, 0, 0, 0, None, "near"),
    ("f16", "same", [700, 20], None, 7, 8, 2, 128, 16, True, 8, 64, 4, 3000, "near"),
    ("bf16", "same", [64, 65], None, 32, 1, 1, 96, 5, False, 0, 3, 0, None, "chain"),
    ("f16", "e4m3", [300, 9], [8, 1], 8, 4, 1, 128, 16, False, 0, 5, 2, 2000, "chain"),
    ("bf16", "int8", [100, 12], None, 12, 2, 2, 80, 48, True, 16, 0, 0, None, "far"),
    # many rows
    ("bf16", "same", [700, 61, 300], [61, 61, 0], 61, 8, 2, 128, 32, True, 0, 0, 0, None, "near"),
    ("f16", "same", [1000, 300], [200, 150], 200, 4, 2, 64, 16, False, 8, 0, 0, 4000, "far"),
    ("bf16", "same", [500], None, 129, 2, 1, 192, 16, False, 0, 40, 300, None, "near"),
    ("f16", "same", [400], None, 300, 1, 1, 80, 16, False, 0, 70, 5, None, "chain"),
    ("bf16", "int8", [900, 100], [64, 100], 100, 4, 1, 128, 16, False, 0, 30, 4, 3000, "near"),
    ("f16", "e4m3", [333], None, 65, 3, 1, 256, 100, True, 0, 0, 0, None, "star"),
    ("bf16", "same", [1030], None, 1024, 1, 1, 64, 16, False, 0, 0, 0, None, "near"),
]


@pytest.mark.parametrize("case", range(len(TREE)))
def test_tree(case):
    dtype, fmt, lens, counts, n, heads, kv, dim, slots, first, gap, window, sinks, hint, kind = TREE[case]
    g = gen(500 + case)
    s = Setup(g, dtype, fmt, lens, counts, n, heads, kv, dim, slots, first, gap)
    s.check(window, sinks, parents_of(g, len(lens), n, kind), hint=hint)


def test_a_chain_is_causal():
    """A tree without branches sees what the last tokens of a row see."""
    g = gen(520)
    for window, sinks in ((0, 0), (20, 3)):
        s = Setup(g, "f16", "same", [300, 41], None, 40, 4, 1, 64, 16)
        a = s.check(window, sinks)
        b = s.check(window, sinks, parents_of(g, 2, 40, "chain"))
        assert np.abs(a[0] - b[0]).max() < 2e-3 and np.abs(a[1] - b[1]).max() < 1e-5


# ---- shared tiles: many rows whose work is cut as for long sequences, or of many sequences ----

FAR = 1 << 20

LONG = [  # dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, heads_first, gap
    ("bf16", "same", [200], None, 200, 4, 1, 64, 16, False, 0),
    ("f16", "same", [300, 70, 5, 0], [33, 33, 5, 1], 33, 2, 2, 128, 16, False, 8),
    ("bf16", "same", [1500, 600], [257, 300], 300, 2, 2, 128, 48, True, 0),
    ("bf16", "same", [1000, 64], None, 65, 3, 3, 96, 33, False, 0),
    ("f16", "same", [700, 200], None, 64, 6, 2, 72, 16, True, 0),
    ("bf16", "same", [513, 100], [70, 100], 100, 4, 2, 192, 16, False, 0),
    ("f16", "same", [450], None, 129, 2, 1, 256, 8, False, 0),
    ("f16", "same", [130], None, 130, 5, 5, 40, 1, False, 0),
    ("bf16", "int8", [777, 200], [300, 133], 300, 5, 1, 80, 48, True, 0),
    ("f16", "e4m3", [1300, 64, 65], None, 100, 8, 2, 128, 16, False, 16),
    ("f16", "int8", [900, 66], [80, 66], 80, 4, 4, 64, 16, False, 0),
    ("bf16", "e4m3", [600], None, 90, 2, 1, 192, 16, True, 0),
    ("f16", "e4m3", [333], None, 140, 1, 1, 96, 1, False, 0),
    ("bf16", "int8", [600, 0, 3], [128, 5, 128], 128, 2, 1, 256, 16, False, 0),
    ("bf16", "e4m3", [700, 33], [40, 33], 40, 1, 1, 112, 100, False, 0),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_long(case):
    dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first, gap = LONG[case]
    s = Setup(gen(700 + case), dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first, gap)
    s.check(hint=FAR)


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 0), (2500, 7), (40, 3)])
@pytest.mark.parametrize("case", range(0, len(LONG), 2))
def test_long_tree(case, window, sinks):
    dtype, fmt, lens, counts, n, heads, kv, dim, slots, first, gap = LONG[case]
    g = gen(720 + case)
    counts = [min(a, b) for a, b in zip(lens, counts or [n] * len(lens))]
    s = Setup(g, dtype, fmt, lens, counts, n, heads, kv, dim, slots, first, gap)
    s.check(window, sinks, parents_of(g, len(lens), n, "near"), hint=FAR)


MANY = [  # dtype, fmt, batch, length, q_len, heads, kv, dim, slots, heads_first, window, sinks
    ("bf16", "same", 14, 260, 160, 8, 8, 64, 16, False, 0, 0),
    ("f16", "same", 17, 400, 130, 8, 8, 128, 16, True, 60, 4),
    ("bf16", "same", 13, 210, 70, 16, 8, 96, 48, False, 64, 64),
    ("f16", "same", 20, 700, 100, 8, 4, 128, 7, False, 500, 1),
    ("bf16", "same", 40, 190, 65, 5, 5, 192, 16, True, 33, 0),
    ("f16", "int8", 18, 300, 130, 8, 8, 64, 16, False, 100, 3),
    ("bf16", "e4m3", 18, 500, 129, 8, 8, 128, 33, True, 90, 90),
    ("bf16", "int8", 15, 280, 100, 12, 6, 80, 16, False, 0, 0),
    ("f16", "e4m3", 40, 150, 65, 5, 5, 256, 16, False, 20, 2),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_sequences(case):
    """More blocks of 32 rows than run at once."""
    dtype, fmt, batch, length, q_len, heads, kv, dim, slots, first, window, sinks = MANY[case]
    g = gen(740 + case)
    lens = [max(0, length - 13 * b) if b % 5 else length for b in range(batch)]
    counts = [0 if b == 3 else max(1, q_len - 11 * (b % 7)) for b in range(batch)]
    s = Setup(g, dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first)
    s.check(window, sinks)
    counts = [min(a, b) for a, b in zip(lens, counts)]
    s = Setup(g, dtype, fmt, lens, counts, q_len, heads, kv, dim, slots, first)
    s.check(window, sinks, parents_of(g, batch, q_len, "far"))


@pytest.mark.parametrize("slots", [1, 2, 16])
@pytest.mark.parametrize("fmt", ["same", "int8"])
def test_more_pages_than_are_looked_up_at_once(fmt, slots):
    """One part of more keys than a thousand pages hold, drafted tokens among them."""
    g = gen(760 + slots)
    n = 1020 * slots + 700
    lens = [n] * 3 + [n - 500] * 2
    for parents, q_len in ((None, 2), (parents_of(g, 5, 8, "near"), 8), (parents_of(g, 5, 30, "near"), 30)):
        s = Setup(g, "f16", fmt, lens, None, q_len, 1, 1, 64, slots)
        s.check(0, 0, parents, hint=100)
        s.check(n - 200, 5, parents, hint=100)


def test_a_long_tree_of_small_pages():
    g = gen(770)
    s = Setup(g, "bf16", "same", [3000], None, 1000, 1, 1, 64, 1)
    s.check(0, 0, parents_of(g, 1, 1000, "near"), hint=100)
    s.check(0, 0, parents_of(g, 1, 1000, "chain"), hint=FAR)
