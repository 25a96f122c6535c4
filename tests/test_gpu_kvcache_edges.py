"""The paged cache's calls at the ends of their ranges.  Tolerances as in
test_gpu_kvcache.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_kvcache as base  # noqa: E402
from gpu_util import require_native  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


# ---- scales ------------------------------------------------------------------------

@pytest.mark.parametrize("prefix, batch", [(0, 3), (90, 3), (1300, 70)])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-38, -3e-39, 1e-45])
def test_scales_near_zero_with_large_scores(scale, prefix, batch):
    """Products of 1e35 and above are still finite in fp32: a scale of 0 makes
    them 0, one of 1e-38 something to weigh by."""
    kv = 120 if prefix == 1300 else 2
    c = ("bf16", batch, 1, kv, kv, 64, 16, prefix, [(7 * i + 5) % 20 for i in range(batch)], False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(51))
    q.mul_(3e17)
    kp.mul_(3e17)
    scale = float(np.float32(scale))
    got, lse = base.attn_run(q, kp, vp, table, lens, rows, 16, prefix, scale, "bf16")
    base.attn_check(got, lse, q, kp, vp, table, lens, rows, 16, prefix, scale, "bf16")


def test_scale_of_zero_keeps_what_is_not_finite():
    """0 times an infinity or a NaN is NaN, in a query and in a key it sees."""
    c = ("f16", 3, 1, 2, 1, 64, 16, 40, [20, 9, 5], False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(52))
    q[0, 0, 1, 3], q[1, 0, 0, 60] = math.inf, math.nan
    kp[int(table[rows[2]][0]), 2, 0, 7] = -math.inf
    got, lse = base.attn_run(q, kp, vp, table, lens, rows, 16, 40, 0.0, "f16")
    bad = np.zeros((3, 1, 2), dtype=bool)
    bad[0, 0, 1] = bad[1, 0, 0] = bad[2] = True
    assert np.array_equal(np.isnan(lse), bad)
    assert np.array_equal(np.isnan(got).all(-1), bad) and np.array_equal(np.isnan(got).any(-1), bad)


# ---- infinite scores -----------------------------------------------------------------

@pytest.mark.parametrize("batch, kv, prefix", [(3, 2, 0), (3, 2, 90), (3, 2, 2000), (80, 500, 300)])
def test_infinite_scores(batch, kv, prefix):
    """All of a query's scores at -inf leave it as one that sees nothing, some
    count as keys that are not there, one at +inf makes it NaN."""
    c = ("bf16", batch, 1, kv, kv, 64, 16, prefix, [20] * batch, False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(53))

    def run():
        return base.attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.125, "bf16")

    q[..., 0].abs_().add_(0.5)                             # head 0 of every key is -inf there
    keep = kp[:, :, 0, 0].clone()
    kp[:, :, 0, 0] = -math.inf
    got, lse = run()
    assert (got[:, 0, 0] == 0).all() and np.isneginf(lse[:, 0, 0]).all()
    assert np.isfinite(got).all() and np.isfinite(lse[:, 0, 1:]).all()
    # the first page of each row's keys alone: as if it were not there
    kp[:, :, 0, 0] = keep
    first = [int(table[r][0]) for r in ([1] if prefix else []) + rows]
    for p in first:
        kp[p, :, 0, 0] = -math.inf
    got, lse = run()
    missing = table.copy()
    missing[:, 0] = -1
    want, lse2 = base.attn_run(q, kp, vp, missing, lens, rows, 16, prefix, 0.125, "bf16")
    with pytest.raises(base.att.TmapError):
        base.att.tile_device_status(base.stream())
    assert np.isfinite(want[:, 0, 0]).all()
    assert np.array_equal(got[:, 0, 0], want[:, 0, 0]) and np.array_equal(lse[:, 0, 0], lse2[:, 0, 0])
    for p in first:
        kp[p, :, 0, 0] = 0.5
    kp[int(table[rows[1]][1]), 2, 1, 0] = math.inf
    got, lse = run()
    assert np.isnan(got[1, 0, 1]).all() and np.isnan(lse[1, 0, 1])
    got[1, 0, 1] = lse[1, 0, 1] = 0
    assert np.isfinite(got).all() and np.isfinite(lse).all()
