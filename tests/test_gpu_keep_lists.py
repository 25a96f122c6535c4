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
