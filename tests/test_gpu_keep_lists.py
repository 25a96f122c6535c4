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
