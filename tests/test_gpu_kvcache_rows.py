"""Rows that are not distinct: what comes out is not said, but every page handed
out is one of the pool's, and nothing else is written."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402

import test_gpu_kvcache as base  # noqa: E402
from gpu_util import require_native, stream  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


@pytest.mark.parametrize("n", [1500, 5000])
def test_extend_of_rows_listed_again_behind_1024_others(n):
    """Row 0 grows to the end of a page among the first 1024 entries and is
    listed again behind them, when it needs a page that was not counted."""
    rows, slots, pages, row_pages = n, 4, 3 * n, 3
    table = torch.full((rows, row_pages), -1, dtype=torch.int32, device="cuda")
    lens, refs = base.ints([0] * rows), base.ints([0] * pages)
    table[0, 0], lens[0], refs[7] = 7, 1, 1
    whole = torch.full((pages + 64,), -5, dtype=torch.int32, device="cuda")    # counts between guards
    whole[32:32 + pages] = refs
    refs = whole[32:32 + pages]
    pt = att.page_table(table, lens, refs, pages, slots)
    who = np.arange(n)
    who[1024:] = 0                                         # again and again
    add = np.ones(n, dtype=np.int32)
    add[:1024] = 4
    add[0] = 3
    add[1024:] = 3
    flag = base.ints([9] * n)
    ws = torch.full((att.page_workspace(pt, n),), 0x7F, dtype=torch.uint8, device="cuda")
    att.page_extend(pt, base.ints(who), base.ints(add), n, flag, ws, stream())
    torch.cuda.synchronize()
    assert set(flag.tolist()) <= {0, 1} and flag[:1024].tolist() == [1] * 1024
    t = table.cpu().numpy()
    assert ((t >= -1) & (t < pages)).all()
    assert (whole[:32] == -5).all() and (whole[-32:] == -5).all()
    counts = refs.cpu().numpy()
    assert set(counts.tolist()) <= {0, 1} and counts.sum() <= 1 + 1023 + (n - 1024)
    # the first 1024 entries are served as they would be alone
    assert (lens[1:1024] == 4).all() and sorted(t[1:1024, 0].tolist()) == [p for p in range(1024) if p != 7]
