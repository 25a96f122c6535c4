"""The paged cache's calls where one round of their loops is not enough:
more entries than a workgroup has threads, more keys than are placed at once,
prefixes in many parts.  Tolerances as in test_gpu_kvcache.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

import test_gpu_kvcache as base  # noqa: E402
from gpu_util import require_native, stream  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


@pytest.mark.parametrize("pages", [9000, 5200])
def test_pages_of_many_rows(pages):
    """2500 entries a call: extends and forks that take pages round after
    round, with 5200 pages running short inside a later round."""
    rows, row_pages, slots = 5000, 6, 4
    rng = np.random.default_rng(pages)
    pool = torch.randint(-999, 999, (pages, slots, 1, 8), generator=base.gen(1)).to(torch.int16).cuda()
    maps = att.tmap_array([base.pool_map(pool, "u16")])
    table = torch.full((rows, row_pages), -1, dtype=torch.int32, device="cuda")
    lens, refs = base.ints([0] * rows), base.ints([0] * pages)
    want = ok.Pages(table.cpu().numpy(), lens.cpu().numpy(), refs.cpu().numpy(), slots, [pool.cpu().numpy()])
    pt = att.page_table(table, lens, refs, pages, slots)
    n = 2500
    ws = torch.empty(att.page_workspace(pt, n), dtype=torch.uint8, device="cuda")
    flag = base.ints([9] * n)

    def check(expect):
        assert flag.cpu().tolist() == expect
        base.same(table, lens, refs, [pool], want)

    who, add = rng.permutation(n), rng.integers(0, 12, n)
    att.page_extend(pt, base.ints(who), base.ints(add), n, flag, ws, stream())
    check(want.extend(who.tolist(), add.tolist()))
    src, dst = rng.integers(0, n, n), n + rng.permutation(n)
    att.page_fork(pt, maps, base.ints(src), base.ints(dst), n, flag, ws, stream())
    check(want.fork(src.tolist(), dst.tolist()))
    who, add = rng.permutation(rows)[:n], rng.integers(0, 5, n)
    att.page_extend(pt, base.ints(who), base.ints(add), n, flag, ws, stream())
    check(want.extend(who.tolist(), add.tolist()))
    assert (pages == 9000) == all(flag.cpu().tolist())
    gone = rng.integers(0, rows, n)
    att.page_free(pt, base.ints(gone), n, stream())
    want.free(gone.tolist())
    base.same(table, lens, refs, [pool], want)


LONG = [  # as ATTN in test_gpu_kvcache.py
    # 80 rows share tiles; 64 heads leave four parts of 384 keys, two placements of addresses each
    ("bf16", 40, 2, 64, 64, 64, 16, 1500, [(5 * i) % 60 for i in range(40)], False, 0),
    # five parts of up to 320 keys, 64 rows a wave's block and a half
    ("f16", 50, 1, 96, 48, 96, 7, 1601, [(7 * i) % 33 for i in range(50)], True, 8),
    # own tokens past one placement, in one part (hint 0) or several
    ("bf16", 2, 1, 4, 2, 128, 48, 70, [1300, 700], True, 0),
    ("f16", 3, 3, 2, 1, 256, 16, 0, [1100, 2, 513], False, 0),
    # products large enough for shared tiles: kv * rows * prefix above 10^7
    ("bf16", 40, 2, 64, 64, 64, 16, 2100, [(5 * i) % 60 for i in range(40)], False, 0),
    ("f16", 50, 1, 96, 48, 96, 7, 2301, [(7 * i) % 33 for i in range(50)], True, 8),
    ("bf16", 70, 1, 16, 16, 200, 48, 9001, [i % 3 for i in range(70)], False, 0),
    # few rows behind a long prefix: each wave has tiles of its own
    ("bf16", 3, 1, 8, 2, 80, 5, 3001, [3, 0, 40], False, 0),
]


@pytest.mark.parametrize("hint", [0, 2000])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_attention_long(case, hint):
    c = LONG[case]
    dtype, slots, prefix = c[0], c[6], c[7]
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(400 + case))
    scale = 1.0 / math.sqrt(c[5])
    got, lse = base.attn_run(q, kp, vp, table, lens, rows, slots, prefix, scale, dtype, hint)
    base.attn_check(got, lse, q, kp, vp, table, lens, rows, slots, prefix, scale, dtype)


@pytest.mark.parametrize("rows_of_queries, kv", [(70, 2), (3, 2), (70, 160)])
def test_bad_pages_in_a_long_prefix(rows_of_queries, kv):
    """Entries of the prefix that are not pages: their keys are not there, for
    every query, and the others' weights do not change."""
    c = ("bf16", rows_of_queries, 1, kv, kv, 64, 16, 1000, [3] * rows_of_queries, False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(9))
    bad = table.copy()
    bad[1, [0, 17, 40]] = [-1, kp.shape[0], 2 ** 31 - 1]
    got, lse = base.attn_run(q, kp, vp, bad, lens, rows, 16, 1000, 0.125, "bf16")
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    # the keys that are left, as a shorter prefix
    keep = [p for i, p in enumerate(table[1][:63]) if i not in (0, 17, 40)]
    short = np.full_like(table, -1)
    short[:] = table
    short[1] = -1
    short[1, :len(keep)] = keep
    base.attn_check(got, lse, q, kp, vp, short, lens, rows, 16, 1000 - 48, 0.125, "bf16")


@pytest.mark.parametrize("batch, kv", [(80, 1), (2, 1), (80, 500)])
def test_values_that_are_not_finite_stay_in_their_column(batch, kv):
    """An infinity among the prefix's values that every query sees: infinite in
    its element, the others as they are."""
    c = ("f16", batch, 1, kv if kv > 1 else 2, kv, 64, 16, 300, [5] * batch, False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(10))
    clean, lse = base.attn_run(q, kp, vp, table, lens, rows, 16, 300, 0.125, "f16")
    vp[int(table[1][7]), 3, :, 11] = math.inf
    got, lse2 = base.attn_run(q, kp, vp, table, lens, rows, 16, 300, 0.125, "f16")
    assert np.isposinf(got[..., 11]).all()
    got[..., 11] = clean[..., 11]
    assert np.array_equal(got, clean) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("batch, kv, prefix", [(80, 500, 300), (3, 2, 300), (3, 2, 2000), (3, 2, 0)])
@pytest.mark.parametrize("where", ["query", "key"])
def test_scores_that_are_not_numbers(batch, kv, prefix, where):
    """A NaN in a query makes all of its scores NaN, one in a key that it sees
    one of them: its result and sum are NaN in either case, the other queries'
    are as they were."""
    c = ("bf16", batch, 1, kv, kv, 64, 16, prefix, [20] * batch, False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(11))
    clean, lse = base.attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.125, "bf16")
    if where == "query":
        q[1, 0, 1, 5] = math.nan
    else:
        kp[int(table[rows[1]][1]), 2, 1, 5] = math.nan
    got, lse2 = base.attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.125, "bf16")
    assert np.isnan(got[1, 0, 1]).all() and np.isnan(lse2[1, 0, 1])
    got[1, 0, 1], lse2[1, 0, 1] = clean[1, 0, 1], lse[1, 0, 1]
    assert np.array_equal(got, clean) and np.array_equal(lse2, lse)
