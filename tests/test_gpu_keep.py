"""GPU parity of page_keep against the oracle: tables, lengths, counts and pools are whole numbers and have to be equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_kvcache import gen, ints, tensor_map  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


class State:
    """Rows of random lengths over pools of random bytes; pools [pages, heads or slots, .., dim]."""

    def __init__(self, g, rows, row_pages, slots, n, dim, heads_first=False, npool=2, codes=False, dtype="u16", gap=0):
        rng = np.random.default_rng(int(torch.randint(0, 1 << 30, (1,), generator=g)))
        self.slots, self.heads_first, self.codes, self.rng, self.dim = slots, heads_first, codes, rng, dim
        pages = rows * row_pages + 2
        lens = rng.integers(0, row_pages * slots + 1, rows).astype(np.int32)
        table = np.full((rows, row_pages), -1, np.int32)
        order, used = rng.permutation(pages), 0
        refs = np.zeros(pages, np.int32)
        for r in range(rows):
            k = -(-int(lens[r]) // slots)
            table[r, :k] = order[used:used + k]
            refs[table[r, :k]] = 1
            used += k
        each = ok.code_rows(slots, dim) if codes else slots
        t = torch.uint8 if codes else {"u8": torch.uint8, "u16": torch.int16, "f32": torch.int32, "f64": torch.int64}[dtype]
        shape = (n, each) if heads_first else (each, n)
        wide = -(-(dim + gap) * t.itemsize // 16) * 16 // t.itemsize
        self.whole = [torch.randint(0, 256, (pages,) + shape + (wide * t.itemsize,), generator=g, dtype=torch.uint8).cuda()
                      .view(t) for _ in range(npool)]
        self.pools = [w[..., :dim] for w in self.whole]
        name = "u8" if codes else dtype
        self.maps = att.tmap_array([tensor_map(self.heads(p), name) for p in self.pools]) if npool else None
        self.table, self.lens, self.refs = ints(table), ints(lens), ints(refs)
        self.pt = att.page_table(self.table, self.lens, self.refs, pages, slots)

    def heads(self, p):
        return p if self.heads_first else p.transpose(1, 2)

    def model(self):
        """The oracle's state: pools as the tokens' bytes [pages, slots, ...], scales behind the codes."""
        flat = []
        for p in self.pools:
            p = self.heads(p).cpu().numpy()                              # [pages, heads, rows, dim]
            x = p[:, :, :self.slots].swapaxes(1, 2)
            if self.codes:
                s = np.ascontiguousarray(p[:, :, self.slots:]).reshape(p.shape[0], p.shape[1], -1)
                s = s[..., :2 * self.slots].reshape(p.shape[0], p.shape[1], self.slots, 2).swapaxes(1, 2)
                x = np.concatenate((x, s), -1)
            flat.append(np.ascontiguousarray(x))
        return ok.Pages(self.table.cpu().numpy(), self.lens.cpu().numpy(), self.refs.cpu().numpy(), self.slots, flat)

    def same_as(self, want):
        got = self.model()
        assert np.array_equal(got.table, want.table) and np.array_equal(got.lens, want.lens)
        assert np.array_equal(got.refs, want.refs)
        assert all(np.array_equal(a, b) for a, b in zip(got.pools, want.pools))

    def lists(self, rows, width):
        """A kept list for each row, from an index that it holds."""
        lens = self.lens.cpu().numpy()
        first = np.array([self.rng.integers(max(0, lens[r] - 2 * width), lens[r] + 1) for r in rows])
        keep, count = np.full((len(rows), width), -7), np.zeros(len(rows), np.int64)
        for i, r in enumerate(rows):
            left = int(lens[r] - first[i])
            count[i] = self.rng.integers(0, min(width, left) + 1)
            keep[i, :count[i]] = np.sort(self.rng.permutation(left)[:count[i]])
        return first, keep, count


def run(s, rows, first, keep, count):
    good = ints(np.full(len(rows), 9))
    att.page_keep(s.pt, s.maps, ints(rows), ints(first), ints(keep), ints(count), len(rows), good, stream())
    return good.tolist()


# rows, row_pages, slots, heads, dim, heads_first, pools, codes, dtype, gap, width
KEEP = [
    (1, 2, 1, 1, 1, False, 1, False, "u8", 0, 2),
    (5, 3, 16, 2, 64, False, 2, False, "u16", 0, 8),
    (4, 9, 7, 3, 77, True, 3, False, "u16", 3, 20),                      # a row's last bytes
    (3, 40, 8, 2, 5, False, 1, False, "f64", 1, 200),                    # more tokens than are placed at once
    (6, 4, 48, 4, 128, True, 17, False, "u8", 0, 33),                    # more than a few pools
    (8, 5, 16, 8, 128, False, 2, True, "u8", 0, 64),
    (3, 6, 5, 3, 80, True, 2, True, "u8", 16, 9),
    (2, 3, 100, 2, 16, False, 1, True, "u8", 0, 150),
    (7, 5, 4, 1, 1, False, 0, False, "u8", 0, 6),                        # the tables alone
    (2, 3, 32, 40, 96, False, 1, False, "f32", 0, 12),                   # more pieces than threads
]


@pytest.mark.parametrize("case", range(len(KEEP)))
def test_keep(case):
    rows, row_pages, slots, n, dim, heads_first, npool, codes, dtype, gap, width = KEEP[case]
    g = gen(300 + case)
    s = State(g, rows, row_pages, slots, n, dim, heads_first, npool, codes, dtype, gap)
    for _ in range(3):
        which = s.rng.permutation(rows)[:max(1, rows - 1)]
        first, keep, count = s.lists(which, width)
        want, whole = s.model(), [w.clone() for w in s.whole]
        expect = want.keep(which, first, keep, count)
        assert expect == [1] * len(which)
        assert run(s, which, first, keep, count) == expect
        s.same_as(want)
        for a, b in zip(s.whole, whole):                                 # between the rows nothing changes
            assert torch.equal(a[..., dim:], b[..., dim:])


def test_keep_refuses_lists():
    """Entries whose list does not ascend or leaves the row are left as they were, beside others that are served."""
    g = gen(320)
    s = State(g, 10, 3, 4, 2, 24)
    lens = np.full(10, 10, np.int32)
    table, refs = np.arange(30, dtype=np.int32).reshape(10, 3), np.ones(32, np.int32)
    s.lens.copy_(ints(lens)), s.table.copy_(ints(table)), s.refs.copy_(ints(refs))
    first = np.array([4, 4, 4, 4, 4, 11, -1, 4, 4, 10])
    keep = np.array([[1, 3], [1, 1], [3, 1], [0, 6], [-1, 2], [0, 1], [0, 1], [0, 1], [0, 1], [0, 0]])
    count = np.array([2, 2, 2, 2, 2, 0, 2, 3, -1, 0])
    want = s.model()
    expect = want.keep(range(10), first, keep, count)
    assert expect == [1, 0, 0, 0, 0, 0, 0, 0, 0, 1]
    assert run(s, np.arange(10), first, keep, count) == expect
    s.same_as(want)


def test_keep_refuses_shared_pages():
    """A page that another row uses too is not written; tokens that stay where they are do not count, nor do pages
    that are only given back."""
    g = gen(321)
    s = State(g, 3, 4, 4, 1, 16)
    s.table.copy_(ints([[0, 1, 2, 3], [0, 1, 4, 5], [6, 7, 8, 9]]))
    s.lens.copy_(ints([16, 16, 16]))
    refs = np.zeros(14, np.int32)
    refs[:10] = [2, 2, 1, 1, 1, 1, 1, 1, 1, 1]
    s.refs.copy_(ints(refs))
    want = s.model()
    args = ([0, 1, 2], [6, 4, 3], [[0, 1, 4], [0, 5, 6], [1, 2, 12]], [3, 3, 3])
    assert want.keep(*args) == [1, 0, 1]                                 # row 0 writes page 2, row 1 page 1
    assert run(s, *(np.array(a) for a in args)) == [1, 0, 1]
    s.same_as(want)
    want = s.model()
    args = ([1], [2], [[0, 1]], [2])                                     # keeps two tokens where they are
    assert want.keep(*args) == [1]
    assert run(s, *(np.array(a) for a in args)) == [1]
    s.same_as(want)


def test_keep_records_what_is_out_of_range():
    g = gen(322)
    s = State(g, 3, 2, 4, 1, 16)
    s.table.copy_(ints([[0, -1], [2, 3], [4, 99]]))
    s.lens.copy_(ints([7, 9, 8]))
    s.refs.fill_(1)
    want = s.model()
    args = ([0, 1, 2, 5, -1], [0] * 5, [[3, 4]] * 5, [2] * 5)            # a page of -1, a row too long, page 99, no rows
    assert want.keep(*args) == [0, 0, 0, 0, 0]
    assert run(s, *(np.array(a) for a in args)) == [0] * 5
    s.same_as(want)
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"


def test_keep_in_a_graph():
    """Rows grow by their drafted tokens and keep some of them, captured once."""
    g = gen(323)
    s = State(g, 4, 8, 4, 2, 32, npool=1)
    n, width, nodes = 4, 3, 6
    s.lens.copy_(ints([9, 0, 4, 17]))
    table = np.full((4, 8), -1, np.int32)
    for r, k in enumerate((3, 0, 1, 5)):
        table[r, :k] = 6 * r + np.arange(k)
    refs = np.zeros(34, np.int32)
    refs[table[table >= 0]] = 1
    s.table.copy_(ints(table)), s.refs.copy_(ints(refs))
    rows, add = ints([2, 0, 3, 1]), ints([nodes] * n)
    first, keep, count = ints([0] * n), ints(np.zeros((n, width))), ints([0] * n)
    grown, good = ints([0] * n), ints([0] * n)
    ws = torch.empty(att.page_workspace(s.pt, n), dtype=torch.uint8, device="cuda")

    def step(st):
        att.page_extend(s.pt, rows, add, n, grown, ws, st)
        att.page_keep(s.pt, s.maps, rows, first, keep, count, n, good, st)

    saved = [t.clone() for t in (s.table, s.lens, s.refs, s.pools[0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(torch.cuda.current_stream().cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for t, old in zip((s.table, s.lens, s.refs, s.pools[0]), saved):
        t.copy_(old)
    for _ in range(4):
        want = s.model()
        base = want.lens[rows.cpu().numpy()]
        kept = np.sort(np.stack([s.rng.permutation(nodes)[:width] for _ in range(n)]), 1)
        some = s.rng.integers(0, width + 1, n)
        first.copy_(ints(base)), keep.copy_(ints(kept)), count.copy_(ints(some))
        assert want.extend(rows.tolist(), [nodes] * n) == [1] * n
        assert want.keep(rows.tolist(), base, kept, some) == [1] * n
        graph.replay()
        torch.cuda.synchronize()
        assert grown.tolist() == [1] * n and good.tolist() == [1] * n
        s.same_as(want)


@pytest.mark.parametrize("entries", [3, 20])
def test_a_row_listed_twice(entries):
    """What is kept is not said, but every page is given back once and the row's length is that of its pages."""
    g = gen(330 + entries)
    s = State(g, 24, 6, 4, 2, 24)
    lens = np.full(24, 22, np.int32)
    table, refs = np.arange(144, dtype=np.int32).reshape(24, 6), np.ones(146, np.int32)
    refs[144:] = 0
    s.lens.copy_(ints(lens)), s.table.copy_(ints(table)), s.refs.copy_(ints(refs))
    rows = np.repeat(np.arange(entries), 2)
    first = s.rng.integers(0, 20, 2 * entries)
    count = s.rng.integers(0, 3, 2 * entries)
    good = run(s, rows, first, np.tile([0, 2], (2 * entries, 1)), np.minimum(count, 22 - first))
    ends, held = s.lens.cpu().numpy(), s.table.cpu().numpy()
    for r in range(24):
        n = -(-int(ends[r]) // 4)
        assert (held[r, :n] >= 0).all() and (held[r, n:] == -1).all()
    assert all(x in (0, 1) for x in good) and (ends[:entries] <= 22).all() and (ends[entries:] == 22).all()
    assert np.array_equal(np.bincount(held[held >= 0], minlength=146), s.refs.cpu().numpy())
    try:                                                                 # an entry that found a page given back may say so
        att.tile_device_status(stream())
    except att.TmapError as e:
        assert e.name == "ERR_PAGE"
