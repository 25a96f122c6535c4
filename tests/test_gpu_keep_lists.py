"""page_keep with lists, rows and pages at the border of what it serves."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_keep import State, run  # noqa: E402
from test_gpu_kvcache import gen, ints  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


def rows_of(n, row_pages, slots, length, npool=2, seed=340):
    """n rows of the same length, each on pages of its own."""
    s = State(gen(seed), n, row_pages, slots, 2, 24, npool=npool)
    used = -(-length // slots)
    table = np.full((n, row_pages), -1, np.int32)
    table[:, :used] = np.arange(n * used).reshape(n, used)
    refs = np.zeros(n * row_pages + 2, np.int32)
    refs[:n * used] = 1
    s.table.copy_(ints(table)), s.lens.copy_(ints(np.full(n, length))), s.refs.copy_(ints(refs))
    return s


@pytest.mark.parametrize("npool", [2, 17])
def test_lists_below_zero(npool):
    """Negative indices that ascend name no token: the entry is left as it was, in one launch and in two."""
    s = rows_of(6, 3, 4, 10, npool)
    first = np.array([0, 4, 9, 0, 0, 2])
    keep = np.array([[-7, -3], [-9, -2], [-2 ** 31, -2 ** 31 + 1], [-1, 0], [-5, 3], [0, 1]])
    want = s.model()
    expect = want.keep(range(6), first, keep, [2] * 6)
    assert expect == [0, 0, 0, 0, 0, 1]
    assert run(s, np.arange(6), first, keep, [2] * 6) == expect
    s.same_as(want)
    att.tile_device_status(stream())


@pytest.mark.parametrize("entries,npool", [(3, 2), (20, 2), (3, 17)])
def test_rows_listed_twice_record_nothing(entries, npool):
    """A page that the row's other entry gave back is no page out of range; run after run, whichever comes first."""
    for k in range(20):
        s = rows_of(24, 6, 4, 22, npool, 350 + k)
        rows = np.repeat(np.arange(entries), 2)
        count = np.tile([2, 0], entries)
        good = run(s, rows, np.full(2 * entries, 3), np.tile([0, 2], (2 * entries, 1)), count)
        assert good == [1] * (2 * entries)
        att.tile_device_status(stream())


@pytest.mark.parametrize("n,npool", [(2, 2), (9, 2), (2, 0), (2, 17)])
def test_missing_pages_are_recorded(n, npool):
    """A row whose pages behind its new end are none is served, and recorded."""
    s = rows_of(n, 6, 4, 22, npool)
    s.table[0, 3], s.table[1, 4] = -1, 6 * n + 2                         # no page, and one behind the last
    want = s.model()
    expect = want.keep(range(n), [5] * n, [[0]] * n, [1] * n)
    assert run(s, np.arange(n), [5] * n, [[0]] * n, [1] * n) == expect == [1] * n
    s.same_as(want)
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"


@pytest.mark.parametrize("npool", [2, 17])
def test_rows_do_not_end_inside_of_shared_pages(npool):
    """Two rows share their first two pages.  One that is cut inside of them would write the other's tokens as it grows
    again: it is left as it was.  Cut at a page's end, or where it ends anyway, it is served."""
    s = rows_of(4, 4, 4, 15, npool)
    s.table[1, :2] = s.table[0, :2]
    s.refs[:2], s.refs[4:6] = 2, 0
    cuts = [([0, 1], [6, 4], [0, 0]), ([0, 1], [1, 5], [3, 2]), ([0, 1], [7, 2], [0, 1]), ([0, 1], [4, 8], [0, 0])]
    got = []
    for rows, first, count in cuts:
        keep = np.tile([0, 1, 2], (2, 1))
        want = s.model()
        expect = want.keep(rows, first, keep, count)
        assert run(s, rows, first, keep, count) == expect
        s.same_as(want)
        got.append(expect)
    assert got == [[0, 1], [1, 0], [0, 0], [1, 0]]
    s.refs[s.table[2, 3]] = 2                                            # an unfinished page that is shared already
    want = s.model()
    args = ([2, 3], [15, 13], [[0], [1]], [0, 1])
    assert want.keep(*args) == [1, 1]
    assert run(s, *(np.array(a) for a in args)) == [1, 1]
    s.same_as(want)


def test_a_fork_that_is_cut_and_grows_leaves_its_twin():
    """A row and its fork share a full page; the fork drops its last tokens.  Whatever the call answers, growing and
    writing the fork afterwards changes no token of the row."""
    s = rows_of(2, 4, 4, 0)
    ws = torch.empty(att.page_workspace(s.pt, 2), dtype=torch.uint8, device="cuda")
    good = ints([0])
    att.page_extend(s.pt, ints([0]), ints([8]), 1, good, ws, stream())
    att.page_fork(s.pt, s.maps, ints([0]), ints([1]), 1, good, ws, stream())
    held = [s.heads(p)[s.table[0, :2].long()].clone() for p in s.pools]
    cut = run(s, [1], [6], [[0]], [0])
    att.page_extend(s.pt, ints([1]), ints([2]), 1, good, ws, stream())
    at = s.lens[1].item() - 1
    for p in s.pools:                                                    # the row's new last token
        s.heads(p)[s.table[1, at // 4].item(), :, at % 4] = 77
    assert cut == [0]
    assert all(torch.equal(s.heads(p)[s.table[0, :2].long()], h) for p, h in zip(s.pools, held))
    att.tile_device_status(stream())
