"""Host side of the calls on pools of 8-bit codes and of page_keep (no GPU):
refusals come before any HIP call, and the oracle's codes are those of torch."""
import numpy as np
import pytest

import async_tensor_tile_amd as att
from oracle import kvcache as ok

from test_kvcache_host import BASE, heads, pool, refused, table


def codes(dim=128, slots=16, n=2, pages=64, rows=None, dtype="u8"):
    rows = att.kv8_rows(slots, dim) if rows is None else rows
    row = -(-dim // 16) * 16
    return att.tmap_encode(dtype, 4, BASE, (dim, rows, n, pages), (row * n, row, row * n * rows), (16, 1, 1, 1))


@pytest.mark.parametrize("slots", [1, 2, 8, 16, 63, 64, 65, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 256])
def test_rows(slots, dim):
    assert att.kv8_rows(slots, dim) == ok.code_rows(slots, dim)


@pytest.mark.parametrize("slots,dim", [(0, 128), (16, 0), (16, 8), (16, 120), (16, 272), (2 ** 31, 128)])
def test_rows_of_none(slots, dim):
    assert att.kv8_rows(slots, dim) == 0


def test_append_refusals():
    r = att.rope_encode(64)

    def call(r=r, q=None, qo=None, k=heads(n=2), v=heads(n=2), fmt="int8", kp=codes(), vp=codes(), pt=table(), rows=BASE,
             at=BASE, pos=BASE):
        return lambda: att.kv8_append(r, q, qo, k, v, fmt, kp, vp, pt, rows, at, pos)

    for c in (call(k=None), call(v=None), call(kp=None), call(vp=None), call(rows=0), call(at=0), call(pos=0),
              call(q=heads()), call(qo=heads()), call(pt=table(t=0))):
        refused(c, "ERR_NULL")
    for fmt in ("same", 3, -1):
        refused(call(fmt=fmt), "ERR_UNSUPPORTED")
    with pytest.raises(ValueError):
        call(fmt="e5m2")()
    refused(call(k=heads(n=2, dtype="f32"), v=heads(n=2, dtype="f32")), "ERR_DTYPE")
    refused(call(kp=heads(n=2)), "ERR_RANK")
    for c in (call(kp=pool(), vp=pool()),                                   # not codes
              call(kp=codes(rows=16), vp=codes(rows=16)),                   # no place for the scales
              call(kp=codes(rows=18), vp=codes(rows=18)), call(vp=codes(n=3)), call(kp=codes(slots=8)),
              call(k=heads(n=3)), call(v=heads(n=2, tokens=15)), call(pt=table(slots=8)), call(pt=table(pages=65)),
              call(kp=codes(dim=64), vp=codes(dim=64)), call(r=att.rope_encode(256)), call(r=att.rope_t()),
              call(q=heads(n=8, dim=64), qo=heads(n=8, dim=64)), call(q=heads(tokens=3), qo=heads(tokens=3)),
              call(k=heads(n=2, dim=72), v=heads(n=2, dim=72), kp=codes(dim=72, rows=17), vp=codes(dim=72, rows=17))):
        refused(c, "ERR_UNSUPPORTED")


def test_read_refusals():
    def call(fmt="e4m3", kp=codes(), vp=codes(), pt=table(), rows=BASE, at=BASE, k=heads(n=2), v=heads(n=2)):
        return lambda: att.kv8_read(fmt, kp, vp, pt, rows, at, k, v)

    for c in (call(kp=None), call(vp=None), call(rows=0), call(at=0), call(k=None), call(v=None), call(pt=table(t=0))):
        refused(c, "ERR_NULL")
    refused(call(k=heads(n=2, dtype="f64"), v=heads(n=2, dtype="f64")), "ERR_DTYPE")
    refused(call(k=pool()), "ERR_RANK")
    for c in (call(fmt="same"), call(fmt=7), call(kp=pool(), vp=pool()), call(kp=codes(rows=16), vp=codes(rows=16)),
              call(v=heads(n=2, dtype="f16")), call(k=heads(n=3)), call(k=heads(n=2, tokens=4)), call(pt=table(slots=8)),
              call(pt=table(pages=63)), call(vp=codes(dim=64)), call(k=heads(n=2, dim=64), v=heads(n=2, dim=64))):
        refused(c, "ERR_UNSUPPORTED")


def test_index_types():
    torch = pytest.importorskip("torch")
    long, odd = torch.zeros(16, dtype=torch.int64), torch.zeros((16, 2), dtype=torch.int32)[:, 0]
    for bad in (long, odd):
        with pytest.raises((TypeError, ValueError)):
            att.kv8_append(None, None, None, heads(n=2), heads(n=2), "int8", codes(), codes(), table(), bad, BASE, BASE)
        with pytest.raises((TypeError, ValueError)):
            att.kv8_read("int8", codes(), codes(), table(), BASE, bad, heads(n=2), heads(n=2))
        with pytest.raises((TypeError, ValueError)):
            att.page_keep(table(), None, bad, BASE, BASE, BASE, 4, BASE, width=4)
    with pytest.raises(ValueError):
        att.page_keep(table(), None, BASE, BASE, torch.zeros((3, 4), dtype=torch.int32), BASE, 4, BASE)
    with pytest.raises(ValueError):
        att.page_keep(table(), None, BASE, BASE, torch.zeros(16, dtype=torch.int32), BASE, 4, BASE)


@pytest.mark.parametrize("short", ["d_rows", "d_from", "d_count", "d_ok"])
def test_keep_takes_a_value_for_each_entry(short):
    torch = pytest.importorskip("torch")
    rows, first, count, good = (torch.zeros(3 if name == short else 4, dtype=torch.int32)
                                for name in ("d_rows", "d_from", "d_count", "d_ok"))
    with pytest.raises(ValueError, match=short):
        att.page_keep(table(), None, rows, first, torch.zeros((4, 4), dtype=torch.int32), count, 4, good)


def test_keep_refusals():
    def call(pt=table(), pools=pool(), rows=BASE, first=BASE, keep=BASE, count=BASE, n=4, good=BASE, width=4):
        return lambda: att.page_keep(pt, pools, rows, first, keep, count, n, good, width=width)

    for c in (call(rows=0), call(first=0), call(keep=0), call(count=0), call(good=0), call(pt=table(lens=0)),
              call(pt=table(refs=0)), call(pt=table(t=0))):
        refused(c, "ERR_NULL")
    for c in (call(pools=pool(slots=8)), call(pools=pool(pages=63)), call(pools=[pool(), pool(n=4)]),
              call(pools=[pool()] * 257), call(pt=table(rows=0)), call(pools=codes(rows=18))):
        refused(c, "ERR_UNSUPPORTED")
    refused(call(pools=heads()), "ERR_RANK")
    call(n=0, rows=0)()
    call(n=0, pools=codes())()
    call(n=0, pools=None)()


def test_pools_of_codes_are_pools():
    """A page of codes has more rows than slots; other types have not."""
    att.page_fork(table(), codes(), BASE, BASE, 0, BASE, BASE, ws_bytes=1 << 20)
    refused(lambda: att.page_fork(table(), pool(slots=17), BASE, BASE, 0, BASE, BASE, ws_bytes=1 << 20),
            "ERR_UNSUPPORTED")


def test_oracle_codes_are_torch_codes():
    torch = pytest.importorskip("torch")
    raw = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(raw.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ok.code_values(raw, "e4m3"), want, equal_nan=True)
    g = np.random.default_rng(1)
    y = g.standard_normal((50, 64)) * np.exp2(g.integers(-20, 20, (50, 1)))
    y[3] = 0
    for fmt in ("int8", "e4m3"):
        s = ok.code_scale(y, fmt)
        assert np.array_equal(torch.from_numpy(s).bfloat16().double().numpy(), s)
        assert (s * ok.LARGEST[fmt] >= np.abs(y).max(-1)).all()
        assert (s * ok.LARGEST[fmt] <= np.abs(y).max(-1) * (1 + 2.0 ** -7)).all()
        c = ok.codes(y, s, fmt)
        z = np.divide(y, s[:, None], out=np.zeros_like(y), where=s[:, None] > 0)
        near = torch.from_numpy(z).float().to(torch.float8_e4m3fn).double().numpy() if fmt == "e4m3" else np.rint(z)
        assert np.array_equal(c, near)
    assert np.isnan(ok.code_scale(np.array([[1.0, np.inf], [np.nan, 0.0]]), "int8")).all()


def test_oracle_keep():
    p = ok.Pages(np.array([[2, 0, 3], [1, 4, -1]], np.int32), np.array([7, 5], np.int32),
                 np.array([1, 1, 1, 1, 2, 0], np.int32), 3, [np.arange(18).reshape(6, 3)])
    # row 0: tokens 2.. are at (2,2) (0,0) (0,1) (0,2) (3,0); keep the second and the fourth
    assert p.keep([0, 1], [2, 3], [[1, 3], [1, 0]], [2, 1]) == [1, 0]     # page 4 is shared: left as it is
    assert p.table.tolist() == [[2, 0, -1], [1, 4, -1]] and p.lens.tolist() == [4, 5]
    assert p.refs.tolist() == [1, 1, 1, 0, 2, 0]
    assert p.pools[0][2].tolist() == [6, 7, 0] and p.pools[0][0].tolist() == [2, 1, 2]
