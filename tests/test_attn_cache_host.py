"""Host side of the attention over the cache (no GPU): refusals come before any
HIP call, and the oracle agrees with small cases worked by hand."""
import numpy as np
import pytest

import async_tensor_tile_amd as att
from oracle import kvcache as ok

from test_kv8_host import codes
from test_kvcache_host import BASE, pool, queries, refused, table


NONE = object()          # an argument that is left out: a module loads no library


def window(q=NONE, kp=NONE, vp=None, fmt="same", pt=None, rows=0, count=0, window=0, sinks=0, hint=64, scale=0.1, o=None,
           lse=0, ws=BASE, n=None):
    q, kp = queries() if q is NONE else q, pool() if kp is NONE else kp
    vp, pt, o = kp if vp is None else vp, pt or table(), queries() if o is None else o
    if n is None:
        n = max(16, att.attn_cache_workspace(q, kp, window, sinks, hint)) if q and kp else 16
    return lambda: att.attn_window(q, kp, vp, fmt, pt, rows, count, window, sinks, hint, scale, o, lse, ws, 0, n)


def tree(q=None, kp=None, fmt="same", pt=None, parent=BASE, hint=64, ws=BASE, n=1 << 40):
    q, kp, pt = q or queries(q_len=5), kp or pool(), pt or table()
    return lambda: att.attn_tree(q, kp, kp, fmt, pt, 0, 0, parent, 0, 0, hint, 0.1, q, 0, ws, 0, n)


def test_window_refusals():
    for c in (window(q=None), window(kp=None, vp=pool()), window(ws=0), window(pt=table(t=0)), window(pt=table(lens=0)),
              lambda: att.attn_window(queries(), pool(), pool(), "same", None, 0, 0, 0, 0, 0, 0.1, queries(), 0, BASE, 0, 64),
              lambda: att.attn_window(queries(), pool(), pool(), "same", table(), 0, 0, 0, 0, 0, 0.1, None, 0, BASE, 0, 64)):
        refused(c, "ERR_NULL")
    refused(window(ws=BASE + 8), "ERR_ALIGN")
    f32 = att.tmap_encode("f32", 4, BASE, (128, 8, 1, 4), (512, 4096, 4096), (4, 1, 1, 1))
    refused(window(q=f32, o=f32, kp=pool(dtype="f32"), n=1 << 20), "ERR_DTYPE")
    refused(window(kp=codes(), fmt="same", n=1 << 20), "ERR_UNSUPPORTED")
    for fmt in (3, -1):
        refused(window(fmt=fmt), "ERR_UNSUPPORTED")
    with pytest.raises(ValueError):
        window(fmt="fp8")()
    q = queries(q_len=8)
    need = att.attn_cache_workspace(q, pool(), 0, 0, 1 << 20)
    assert need > 16
    for c in (window(q=queries(dtype="f16")), window(o=queries(n=4)), window(kp=pool(slots=8)), window(kp=pool(pages=63)),
              window(kp=pool(dim=64)), window(vp=pool(n=4)), window(q=queries(n=7), o=queries(n=7), kp=pool(n=2)),
              window(scale=float("nan")), window(scale=3e38), window(fmt="int8", kp=pool()),
              window(fmt="int8", kp=codes(rows=16)), window(fmt="e4m3", kp=codes(slots=8)),
              window(q=q, o=q, hint=1 << 20, n=need - 1)):
        refused(c, "ERR_UNSUPPORTED")
    assert att.attn_cache_workspace(queries(), pool(dim=64), 0, 0, 64) == 0
    assert att.attn_cache_workspace(queries(), None, 0, 0, 64) == 0


def test_tree_refusals():
    refused(tree(parent=0), "ERR_NULL")
    refused(tree(q=queries(q_len=1025)), "ERR_UNSUPPORTED")
    refused(tree(kp=pool(slots=8)), "ERR_UNSUPPORTED")
    refused(tree(ws=BASE + 4), "ERR_ALIGN")
    refused(tree(kp=codes()), "ERR_UNSUPPORTED")


def test_more_than_one_launch():
    """2^24 - 1 workgroups of 256 threads."""
    p = pool(n=512)
    assert att.attn_cache_workspace(queries(n=512, batch=32760), p, 0, 0, 0) > 0
    assert att.attn_cache_workspace(queries(n=512, batch=32768), p, 0, 0, 0) == 0
    refused(window(q=queries(n=512, batch=32768), o=queries(n=512, batch=32768), kp=p, pt=table(rows=40000), n=1 << 40),
            "ERR_UNSUPPORTED")
    assert att.attn_cache_workspace(queries(n=64, q_len=65535, batch=600), pool(n=1), 0, 0, 0) == 0   # rows beyond 31 bits


def test_workspace_follows_the_window():
    q, p = queries(q_len=1, batch=1), pool()
    short, far = (att.attn_cache_workspace(q, p, w, 4, 1 << 20) for w in (200, 0))
    assert 0 < short < far


def test_index_types():
    torch = pytest.importorskip("torch")
    long = torch.zeros(16, dtype=torch.int64)
    for c in (window(rows=long), window(count=long), tree(parent=long)):
        with pytest.raises(TypeError):
            c()
    with pytest.raises(TypeError):
        window(lse=torch.zeros(4, dtype=torch.float64))()


def test_oracle_windows():
    got = ok.causal_sees(6, 3, 2, 1).astype(int).tolist()
    assert got == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert ok.causal_sees(2, 3, 0, 0).astype(int).tolist() == [[0, 0], [1, 0], [1, 1]]
    # context of 3, then nodes 0 <- 1, 0 <- 2, context <- 3, 2 <- 4
    got = ok.tree_sees(8, [-1, 0, 0, -1, 2], 0, 0).astype(int).tolist()
    assert got == [[1, 1, 1, 1, 0, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 1, 0, 0], [1, 1, 1, 0, 0, 0, 1, 0],
                   [1, 1, 1, 1, 0, 1, 0, 1]]
    got = ok.tree_sees(8, [-1, 0, 0, -1, 2], 2, 1).astype(int).tolist()
    assert got[4] == [1, 0, 0, 0, 0, 1, 0, 1] and got[3] == [1, 0, 1, 0, 0, 0, 1, 0]


def test_oracle_attention():
    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    k, v = np.array([[[1.0, 0.0]], [[0.0, 1.0]]]), np.array([[[2.0, 4.0]], [[np.nan, 6.0]]])
    o, lse, _, _, seen = ok.attend(q, k, v, np.array([[True, False], [False, False]]), 1.0)
    assert o[0, 0].tolist() == [2.0, 4.0] and o[1, 0].tolist() == [0.0, 0.0]
    assert lse[0, 0] == 1.0 and np.isneginf(lse[1, 0]) and seen[:, 0].tolist() == [1, 0]


def test_workgroups_of_a_call():
    """Few rows: a part of partial results for each workgroup, [dim rounded up, 32] sums and 32 pairs of 8 bytes."""
    most = 0
    for batch in (1, 2, 3, 7, 16, 31, 32, 40, 63, 64, 65, 100, 128, 129, 200, 300, 511, 512, 513, 700, 5000):
        for kv in (1, 2, 8):
            for group in (1, 4, 32):
                for hint in (0, 500, 2047, 2048, 3000, 8192, 20000, 1 << 20, 2 ** 32 - 1):
                    for window in (0, 4096):
                        got = att.attn_cache_workspace(queries(dim=64, n=kv * group, batch=batch), pool(dim=64, n=kv),
                                                       window, 4, hint)
                        parts = (got - 16) // (64 * 32 * 4 + 32 * 8)
                        assert (got - 16) % (64 * 32 * 4 + 32 * 8) == 0
                        units = batch * kv
                        assert parts <= max(4 * units, 1280) and parts % units == 0
                        most = max(most, parts / units if units > 256 else 0)
    assert most > 1                                                      # more than one a unit, and than 512 in all
