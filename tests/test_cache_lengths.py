"""Tensors with fewer values than a call of the paged cache reads or writes are
refused before the library is called (no GPU): the device would read or write
behind them."""
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att

from test_kv8_host import codes
from test_kvcache_host import BASE, heads, pool, queries, refused, table


def values(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def short(call, name):
    """`call` with one value too few of each argument is refused, by its name."""
    with pytest.raises(ValueError, match=name):
        call()


@pytest.mark.parametrize("dims", [(128, 8, 1, 4), (96, 5, 77, 3), (8, 1, 1024, 1)])
def test_map_dims(dims):
    dim, n, q_len, batch = dims
    def of(m):
        return m.dim0, m.dim1, m.dim2, m.dim3, m.dim4

    assert of(queries(dim, n, q_len, batch)) == (*dims, 1)
    assert of(att.tmap_array([queries(), queries(dim, n, q_len, batch)])[1]) == (*dims, 1)
    assert of(heads(128, 7, 2 ** 31 - 1)) == (128, 7, 2 ** 31 - 1, 1, 1)


# what a call of 4 sequences with 3 queries of 8 heads takes
WINDOW = {"d_rows": 4, "d_count": 4, "d_lse": 96}
TREE = dict(WINDOW, d_parent=12)


def window(**n):
    v = {k: values(n.get(k, x), torch.float32 if k == "d_lse" else torch.int32) for k, x in WINDOW.items()}
    att.attn_window(queries(q_len=3), pool(), pool(), "same", table(), v["d_rows"], v["d_count"], 0, 0, 64, 0.1,
                    queries(q_len=3), v["d_lse"], 0)


def tree(**n):
    v = {k: values(n.get(k, x), torch.float32 if k == "d_lse" else torch.int32) for k, x in TREE.items()}
    att.attn_tree(queries(q_len=3), pool(), pool(), "same", table(), v["d_rows"], v["d_count"], v["d_parent"], 0, 0, 64, 0.1,
                  queries(q_len=3), v["d_lse"], 0)


@pytest.mark.parametrize("call,sizes", [(window, WINDOW), (tree, TREE)])
def test_attention(call, sizes):
    refused(call, "ERR_NULL")                                            # enough of all: the missing workspace is next
    refused(lambda: call(**{k: 5 * n for k, n in sizes.items()}), "ERR_NULL")
    for name, n in sizes.items():
        short(lambda: call(**{name: n - 1}), name)


def test_parents_of_any_shape():
    for t in (torch.zeros((4, 3), dtype=torch.int32), torch.zeros((2, 6), dtype=torch.int32)):
        refused(lambda: att.attn_tree(queries(q_len=3), pool(), pool(), "same", table(), None, None, t, 0, 0, 64, 0.1,
                                      queries(q_len=3), None, 0), "ERR_NULL")


@pytest.mark.parametrize("name", ["d_rows", "d_at", "d_pos"])
def test_append(name):
    def call(n, r=att.rope_encode(64), d_pos=None):
        rows, at, pos = (values(n if name == k else 16) for k in ("d_rows", "d_at", "d_pos"))
        att.kv8_append(r, None, None, heads(n=2), heads(n=2), "int8", codes(), codes(), None, rows, at,
                       pos if d_pos is None else d_pos)

    refused(lambda: call(16), "ERR_NULL")                                # no table
    short(lambda: call(15), name)
    if name == "d_pos":                                                  # not read without a plan
        refused(lambda: call(16, None, values(0)), "ERR_NULL")


@pytest.mark.parametrize("name", ["d_rows", "d_at"])
def test_read(name):
    def call(n):
        rows, at = (values(n if name == k else 16) for k in ("d_rows", "d_at"))
        att.kv8_read("int8", codes(), codes(), None, rows, at, heads(n=2), heads(n=2))

    refused(lambda: call(16), "ERR_NULL")
    short(lambda: call(15), name)


@pytest.mark.parametrize("n", [-1, -2 ** 31, 2 ** 32])
def test_keep_counts(n):
    with pytest.raises(ValueError, match="n has"):
        att.page_keep(table(), None, BASE, BASE, torch.zeros((4, 4), dtype=torch.int32), BASE, n, BASE)
    with pytest.raises(ValueError, match="width has"):
        att.page_keep(table(), None, BASE, BASE, BASE, BASE, 4, BASE, width=n)


# ---- the calls on pages of 16 bits and behind a shared prefix --------------------------


def test_rope():
    r, x = att.rope_encode(64), heads()
    refused(lambda: att.rope_apply(r, x, heads(n=9), values(16)), "ERR_UNSUPPORTED")
    short(lambda: att.rope_apply(r, x, heads(n=9), values(15)), "d_pos")


@pytest.mark.parametrize("name", ["d_rows", "d_at", "d_pos"])
def test_append_same(name):
    def call(n, r=att.rope_encode(64), d_pos=None):
        rows, at, pos = (values(n if name == k else 16) for k in ("d_rows", "d_at", "d_pos"))
        att.rope_append(r, None, None, heads(n=2), heads(n=2), pool(), pool(), None, rows, at,
                        pos if d_pos is None else d_pos)

    refused(lambda: call(16), "ERR_NULL")
    short(lambda: call(15), name)
    if name == "d_pos":
        refused(lambda: call(16, None, values(0)), "ERR_NULL")


def test_pages():
    four, three = values(4), values(3)
    ws = values(1 << 12)
    t = table(lens=0)                                                    # refused once the library is called
    for a, b, name in ((three, four, "d_src"), (four, three, "d_dst")):
        short(lambda: att.page_copy(pool(), a, b, 4), name)
        short(lambda: att.page_fork(t, None, a, b, 4, four, ws), name)
    for a, b, c, name in ((three, four, four, "d_rows"), (four, three, four, "d_add"), (four, four, three, "d_ok")):
        short(lambda: att.page_extend(t, a, b, 4, c, ws), name)
    short(lambda: att.page_fork(t, None, four, four, 4, three, ws), "d_ok")
    short(lambda: att.page_free(t, three, 4), "d_rows")
    short(lambda: att.page_compact(t, t, None, values(0), ws), "d_used")
    refused(lambda: att.page_extend(t, four, four, 4, four, ws), "ERR_NULL")
    refused(lambda: att.page_fork(t, None, four, four, 4, four, ws), "ERR_NULL")
    refused(lambda: att.page_free(t, four, 4), "ERR_NULL")
    refused(lambda: att.page_compact(table(refs=0), t, None, values(1), ws), "ERR_NULL")
    for call in (lambda: att.page_copy(pool(), BASE, BASE, -1), lambda: att.page_free(t, BASE, -1),
                 lambda: att.page_extend(t, BASE, BASE, -1, BASE, ws), lambda: att.page_workspace(t, -1),
                 lambda: att.page_fork(t, None, BASE, BASE, 2 ** 32, BASE, ws)):
        short(call, "n has")


def test_shared_prefix():
    def call(rows=4, lse=96):
        att.attn_shared_prefix(queries(q_len=3), pool(), pool(), table(), 0, 0, values(rows), 64, 0.1, queries(q_len=3),
                               values(lse, torch.float32), 0)

    refused(call, "ERR_NULL")
    short(lambda: call(rows=3), "d_rows")
    short(lambda: call(lse=95), "d_lse")
