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
    assert att._dims(queries(dim, n, q_len, batch)) == (*dims, 1)
    assert att._dims(att.tmap_array([queries(), queries(dim, n, q_len, batch)])[1]) == (*dims, 1)
    assert att._dims(heads(128, 7, 2 ** 31 - 1)) == (128, 7, 2 ** 31 - 1, 1, 1)


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
