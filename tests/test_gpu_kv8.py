"""GPU parity of the calls on pools of 8-bit codes against the 64-bit oracle.

A value's code and scale have to be the oracle's, bit for bit: the elements
have 8 or 11 significant bits and the scale 8, so a quotient that is not on the
border between two codes is at least 2^-20 of itself away from it, and a
correctly rounded fp32 quotient stays on its side.  A key is rotated in fp32
first, off by at most 2^-21 of the magnitudes in its pair (angle, function,
magnitude; the roundings are below that), so its scale is the oracle's within
that and one step of bf16, and its code times its own scale is within half a
code's step of the exact key, plus that error and one rounding of the quotient.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_kvcache import TORCH, f64, gen, ints, padded, rope_limit, tensor_map  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


class Cache:
    """Two pools of random bytes, a table with some of its entries unused."""

    def __init__(self, rows, row_pages, slots, n, dim, heads_first, g, extra=3, gap=0):
        self.slots, self.n, self.dim, self.heads_first = slots, n, dim, heads_first
        self.pages = rows * row_pages + extra
        shape = (n, ok.code_rows(slots, dim)) if heads_first else (ok.code_rows(slots, dim), n)
        self.whole = [torch.randint(0, 256, (self.pages,) + shape + (dim + gap,), generator=g, dtype=torch.uint8).cuda()
                      for _ in "kv"]
        self.pools = [w[..., :dim] for w in self.whole]
        self.maps = [tensor_map(p if heads_first else p.transpose(1, 2), "u8") for p in self.pools]
        table = torch.randperm(self.pages, generator=g)[:rows * row_pages].view(rows, row_pages).int()
        self.table = table.cuda()
        self.pt = att.page_table(self.table, None, None, self.pages, slots)

    def split(self, i, fmt):
        """Codes [pages, heads, slots, dim] and scales of pool i, on the host."""
        p = self.pools[i].cpu().numpy()
        return ok.split_codes(p if self.heads_first else p.transpose(0, 2, 1, 3), self.slots, fmt)

    def places(self, rows, at):
        t = self.table.cpu().numpy()
        return t[rows, at // self.slots], at % self.slots


def spots(rows, row_tokens, tokens, g):
    """Distinct (row, index) pairs."""
    flat = torch.randperm(rows * row_tokens, generator=g)[:tokens].numpy()
    return flat // row_tokens, flat % row_tokens


# dtype, fmt, tokens, q heads, kv heads, dim, rot, layout, slots, heads_first, gap
APPEND = [
    ("bf16", "int8", 1, 4, 1, 64, 64, "half", 16, False, 0),
    ("f16", "e4m3", 7, 6, 3, 128, 128, "half", 16, True, 0),
    ("bf16", "e4m3", 33, 8, 2, 80, 20, "half", 8, False, 16),          # halves that are not whole chunks
    ("f16", "int8", 9, 5, 5, 96, 62, "interleaved", 48, True, 0),
    ("bf16", "int8", 21, 0, 4, 256, 256, "interleaved", 1, False, 0),   # no queries
    ("f16", "e4m3", 65, 3, 1, 16, 2, "half", 100, True, 32),
    ("bf16", "e4m3", 12, 2, 2, 240, 240, "half", 7, False, 0),
    ("f16", "int8", 5, 64, 64, 48, 0, "half", 64, False, 0),            # not rotated
    ("bf16", "int8", 1030, 4, 2, 112, 16, "half", 16, True, 0),         # two tokens a workgroup
    ("f16", "e4m3", 1027, 40, 8, 192, 192, "interleaved", 33, False, 0),
    ("bf16", "e4m3", 4100, 32, 8, 128, 128, "half", 16, False, 0),      # more than the L2s hold
    ("f16", "int8", 4100, 32, 8, 128, 34, "half", 48, True, 16),
    ("f16", "e4m3", 2051, 64, 2, 144, 144, "interleaved", 16, False, 0),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case):
    dtype, fmt, tokens, hq, n, dim, rot, layout, slots, heads_first, gap = APPEND[case]
    g = gen(100 + case)
    rows = 3
    row_pages = -(-(tokens + 5) // slots)
    c = Cache(rows, row_pages, slots, n, dim, heads_first, g, gap=gap)
    _, k = padded((tokens, n, dim), dtype, gap, g)
    _, v = padded((tokens, n, dim), dtype, gap + 8, g)
    row, at = spots(rows, row_pages * slots, tokens, g)
    pos = torch.randint(-1000, 1 << 20, (tokens,), generator=g).numpy()
    d_row, d_at, d_pos = ints(row), ints(at), ints(pos)
    args = (10000.0, "none", 1.0, 0, 1.0, 32.0)
    plan = att.rope_encode(rot, layout, *args, 1.25) if rot else None
    before = [c.split(i, fmt) for i in (0, 1)]
    mk, mv, mq = tensor_map(k, dtype), tensor_map(v, dtype), None
    if hq:
        _, q = padded((tokens, hq, dim), dtype, gap, g)
        q_old = f64(q)
        mq = tensor_map(q, dtype)                                        # turned in place
    att.kv8_append(plan, mq, mq, mk, mv, fmt, *c.maps, c.pt, d_row, d_at, d_pos if rot else None, stream())
    thetas = ok.rope_thetas(rot, *args) if rot else []
    slack = np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -52
    if hq:
        want, size = ok.rope(q_old, pos, thetas, layout, 1.25) if rot else (q_old, np.abs(q_old))
        assert (np.abs(f64(q) - want) <= rope_limit(want, size, dtype) + size * slack).all()
    page, slot = c.places(row, at)
    # values: the oracle's codes and scales
    code, scale = c.split(1, fmt)
    y = f64(v)
    s = ok.code_scale(y, fmt)
    assert np.array_equal(scale[page, :, slot], s)
    assert np.array_equal(code[page, :, slot], ok.codes(y, s, fmt))
    # keys
    code, scale = c.split(0, fmt)
    y, size = ok.rope(f64(k), pos, thetas, layout, 1.25) if rot else (f64(k), np.abs(f64(k)))
    off = size * (2.0 ** -21 + slack) if rot else 0 * size
    s, top = scale[page, :, slot], np.abs(y).max(-1) / ok.LARGEST[fmt]
    assert (s >= top - off.max(-1)).all() and (s <= (top + off.max(-1)) * (1 + 2.0 ** -7) * (1 + 2.0 ** -23)).all()
    z = y / s[..., None]
    step = s[..., None] * ok.code_step(z * (1 + 2.0 ** -20), fmt)
    assert (np.abs(code[page, :, slot] * s[..., None] - y) <= step / 2 + off + 2.0 ** -24 * np.abs(y)).all()
    # everything else is as it was
    rest = np.ones((c.pages, slots), bool)
    rest[page, slot] = False
    for i in (0, 1):
        now = c.split(i, fmt)
        for a, b in zip(now, before[i]):
            a, b = a.swapaxes(1, 2)[rest], b.swapaxes(1, 2)[rest]
            assert np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_special_values(dtype, fmt):
    """Zeros, infinities, NaN, the smallest and largest numbers, borders between codes."""
    g = gen(5)
    n, dim, slots = 2, 32, 4
    c = Cache(1, 4, slots, n, dim, False, g)
    big, tiny = torch.finfo(TORCH[dtype]).max, {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dtype]
    v = torch.zeros(12, n, dim)
    v[1] = torch.randn(n, dim, generator=g)
    v[1, 0, 3] = float("inf")
    v[2] = torch.randn(n, dim, generator=g)
    v[2, 1, 31] = float("nan")
    v[3] = big
    v[3, :, 1] = -big
    v[4] = tiny * torch.randint(-3, 4, (n, dim), generator=g)
    v[5, :, 7] = -tiny
    v[6] = torch.arange(-16, 16) / 2                                     # halves of the largest code over 2^k
    v[6, :, 0] = ok.LARGEST[fmt] / 8
    v[7] = torch.arange(-16, 16) + 0.5
    v[7, :, 0] = ok.LARGEST[fmt]
    v[8, 0, 0] = float("-inf")
    v[9] = -0.0
    v[10] = torch.randn(n, dim, generator=g) * 2.0 ** -13
    v[11] = torch.arange(32) * 0.5
    v[11, :, 0] = ok.LARGEST[fmt]
    v = v.to(TORCH[dtype]).cuda()
    k = v.flip(0).contiguous()
    rows, at = np.zeros(12, np.int64), np.arange(12)
    att.kv8_append(None, None, None, tensor_map(k, dtype), tensor_map(v, dtype), fmt, *c.maps, c.pt, ints(rows), ints(at),
                   None, stream())
    page, slot = c.places(rows, at)
    for i, y in enumerate((f64(k), f64(v))):
        code, scale = c.split(i, fmt)
        s = ok.code_scale(y, fmt)
        assert np.array_equal(scale[page, :, slot], s, equal_nan=True)
        assert np.array_equal(code[page, :, slot], ok.codes(y, s, fmt))
    back = [torch.zeros_like(v) for _ in "kv"]
    att.kv8_read(fmt, *c.maps, c.pt, ints(rows), ints(at), *(tensor_map(b, dtype) for b in back), stream())
    assert torch.isnan(back[1][1, 0]).all() and torch.isnan(back[1][2, 1]).all() and torch.isnan(back[1][8, 0]).all()
    assert torch.isfinite(back[1][1, 1]).all() and (back[1][0] == 0).all()


def test_append_leaves_out_what_has_no_place():
    """Padding is silent; a row, index or page out of range is recorded and nothing else is written."""
    g = gen(6)
    c = Cache(2, 2, 4, 1, 16, False, g)
    c.table[1, 1] = -1
    before = [p.clone() for p in c.pools]
    k = torch.randn(6, 1, 16, generator=g).bfloat16().cuda()
    m = tensor_map(k, "bf16")
    att.kv8_append(None, None, None, m, m, "int8", *c.maps, c.pt, ints([-1] * 6), ints([0] * 6), None, stream())
    att.tile_device_status(stream())
    att.kv8_append(None, None, None, m, m, "int8", *c.maps, c.pt, ints([2, 1, 1, 0, 0, -5]), ints([0, 5, 8, -1, 99, 0]),
                   None, stream())
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    assert all(torch.equal(a, b) for a, b in zip(before, c.pools))


# dtype, fmt, tokens, kv heads, dim, slots, heads_first, gap
READ = [
    ("f32", "int8", 1, 1, 16, 1, False, 0),
    ("f16", "int8", 9, 3, 128, 16, True, 0),
    ("bf16", "e4m3", 100, 8, 96, 48, False, 16),
    ("f32", "e4m3", 513, 5, 80, 7, True, 16),
    ("bf16", "int8", 2049, 64, 256, 100, False, 0),
    ("f16", "e4m3", 8, 2, 48, 64, True, 32),
]


@pytest.mark.parametrize("case", range(len(READ)))
def test_read(case):
    """A code has at most 8 significant bits and the scale 8: the product is exact in fp32 and rounded once."""
    dtype, fmt, tokens, n, dim, slots, heads_first, gap = READ[case]
    g = gen(200 + case)
    row_pages = -(-(tokens + 5) // slots)
    c = Cache(2, row_pages, slots, n, dim, heads_first, g, gap=gap)
    row, at = spots(2, row_pages * slots, tokens, g)
    row[::7] = -1
    whole = [torch.full((tokens, n, dim + 16), 7.0, dtype=TORCH[dtype], device="cuda") for _ in "kv"]
    out = [w[..., :dim] for w in whole]
    # scales a cache would hold: random bytes are no numbers
    for p in c.pools:
        s = torch.rand((c.pages, n, slots), generator=g).bfloat16()
        tail = torch.zeros((c.pages, n, (ok.code_rows(slots, dim) - slots) * dim), dtype=torch.uint8)
        tail[..., :2 * slots] = s.view(torch.uint8)
        tail = tail.view(c.pages, n, -1, dim).cuda()
        (p if heads_first else p.transpose(1, 2))[:, :, slots:] = tail
    att.kv8_read(fmt, *c.maps, c.pt, ints(row), ints(at), *(tensor_map(o, dtype) for o in out), stream())
    page, slot = c.places(row, at)
    for i in (0, 1):
        code, scale = c.split(i, fmt)
        want = code[page, :, slot] * scale[page, :, slot][..., None]
        want[row < 0] = 7.0
        want = torch.from_numpy(want).float().to(TORCH[dtype])
        assert torch.equal(out[i].cpu().nan_to_num(1e4), want.nan_to_num(1e4))
        assert (whole[i][..., dim:] == 7.0).all()


def test_read_leaves_out_what_is_not_there():
    g = gen(7)
    c = Cache(2, 2, 4, 1, 16, True, g)
    c.table[0, 0] = c.pages
    out = torch.full((5, 1, 16), 3.0, dtype=torch.float16, device="cuda")
    m = tensor_map(out, "f16")
    att.kv8_read("e4m3", *c.maps, c.pt, ints([0, 2, 1, 1, -1]), ints([0, 0, 8, -1, 0]), m, m, stream())
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    assert (out == 3.0).all()


@pytest.mark.parametrize("heads_first", [False, True])
def test_pages_of_codes_move_whole(heads_first):
    """Forked, copied and compacted pages carry their scales."""
    g = gen(8)
    slots, n, dim, pages = 6, 2, 32, 20
    c = Cache(2, 4, slots, n, dim, heads_first, g, extra=12)
    table = torch.full((4, 4), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = ints([5, 17, 9])
    lens, refs = ints([15, 0, 0, 0]), torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[ints([5, 17, 9]).long()] = 1
    pt = att.page_table(table, lens, refs, pages, slots)
    ws = torch.empty(att.page_workspace(pt, 4), dtype=torch.uint8, device="cuda")
    good, used = ints([0, 0]), ints([0])
    maps = att.tmap_array(c.maps)
    heads = [p if heads_first else p.transpose(1, 2) for p in c.pools]

    def held(row):
        t = table[row, :3].long()
        return [h[t].clone() for h in heads]

    first = held(0)
    att.page_fork(pt, maps, ints([0, 0]), ints([1, 2]), 2, good, ws, stream())
    assert good.tolist() == [1, 1]
    for r in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(first, held(r)))
    att.page_copy(maps, ints([5]), ints([19]), 1, stream())
    assert all(torch.equal(h[5], h[19]) for h in heads)
    att.page_compact(pt, pt, maps, used, ws, stream())
    assert used.item() == 5 and int(table.max()) == 4
    for r in (0, 1, 2):
        assert all(torch.equal(a, b) for a, b in zip(first, held(r)))


def test_append_and_read_in_a_graph():
    """Captured once and replayed with other tokens, places and rows, the program's own work between."""
    g = gen(9)
    tokens, n, dim, slots = 16, 2, 64, 8
    c = Cache(2, 8, slots, n, dim, False, g)
    k, v, q = (torch.zeros((tokens, h, dim), dtype=torch.bfloat16, device="cuda") for h in (n, n, 4))
    kb, vb, qo = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
    d_row, d_at, d_pos = (ints(np.zeros(tokens)) for _ in range(3))
    plan = att.rope_encode(dim)
    maps = [tensor_map(t, "bf16") for t in (q, qo, k, v)]
    back = [tensor_map(t, "bf16") for t in (kb, vb)]

    def step(st):
        att.kv8_append(plan, *maps, "e4m3", *c.maps, c.pt, d_row, d_at, d_pos, st)
        att.kv8_read("e4m3", *c.maps, c.pt, d_row, d_at, *back, st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(torch.cuda.current_stream().cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        row, at = spots(2, 8 * slots, tokens, g)
        for t, x in ((k, n), (v, n), (q, 4)):
            t.copy_(torch.randn((tokens, x, dim), generator=g).bfloat16())
        d_row.copy_(ints(row)), d_at.copy_(ints(at)), d_pos.copy_(ints(at + 100 * i))
        graph.replay()
        got = [t.clone() for t in (qo, kb, vb)]
        torch.cuda.synchronize()
        for t in (qo, kb, vb):
            t.zero_()
        step(stream())
        assert all(torch.equal(a, b) for a, b in zip(got, (qo, kb, vb)))
        s = torch.from_numpy(ok.code_scale(f64(v), "e4m3"))
        assert torch.equal(vb.cpu(), torch.from_numpy(ok.codes(f64(v), s.numpy(), "e4m3") * s.numpy()[..., None]).bfloat16())
