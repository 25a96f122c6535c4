"""Host side of the paged cache's calls (no GPU): refusals come before any
HIP call, and the oracle agrees with small cases worked by hand."""
import math

import numpy as np
import pytest

import async_tensor_tile_amd as att
from oracle import kvcache as ok

BASE = 0x7F0000000000   # a 16-byte aligned stand-in address; nothing here reaches a kernel


def heads(dim=128, n=8, tokens=16, dtype="bf16", base=BASE, **kw):
    e = att.ESIZE[dtype]
    row = -(-dim * e // 16) * 16
    return att.tmap_encode(dtype, 3, base, (dim, n, tokens), (row, row * n), (16 // e, 1, 1), **kw)


def queries(dim=128, n=8, q_len=1, batch=4, dtype="bf16"):
    return att.tmap_encode(dtype, 4, BASE, (dim, n, q_len, batch), (dim * 2, dim * n * 2, dim * n * q_len * 2),
                           (8, 1, 1, 1))


def pool(dim=128, slots=16, n=2, pages=64, dtype="bf16", **kw):
    e = att.ESIZE[dtype]
    row = dim * e
    return att.tmap_encode(dtype, 4, BASE, (dim, slots, n, pages), (row * n, row, row * n * slots), (16 // e, 1, 1, 1),
                           **kw)


def table(rows=8, row_pages=8, pages=64, slots=16, pitch=0, t=BASE, lens=BASE, refs=BASE):
    return att.page_table(t, lens, refs, pages, slots, rows, row_pages, pitch)


def refused(call, name):
    with pytest.raises(att.TmapError) as e:
        call()
    assert e.value.name == name


@pytest.mark.parametrize("args", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_dim=64, layout=2),
                                  dict(rot_dim=64, scaling=4), dict(rot_dim=64, base=0.0),
                                  dict(rot_dim=64, base=float("nan")), dict(rot_dim=64, base=float("inf")),
                                  dict(rot_dim=64, scaling="linear", factor=0.0),
                                  dict(rot_dim=64, scaling="base", factor=float("nan")),
                                  dict(rot_dim=64, scaling="ramp", factor=2.0),
                                  dict(rot_dim=64, scaling="ramp", factor=2.0, original_len=10, slow=4.0, fast=4.0),
                                  dict(rot_dim=64, magnitude=float("inf"))])
def test_rope_encode_refusals(args):
    refused(lambda: att.rope_encode(**args), "ERR_UNSUPPORTED")


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp"])
@pytest.mark.parametrize("rot", [2, 6, 64, 256])
def test_rope_plan_holds_the_frequencies(rot, scaling):
    """The plan's first rot / 2 doubles are turns per position."""
    r = att.rope_encode(rot, "half", 500000.0, scaling, 8.0, 4096, 1.0, 4.0)
    got = np.frombuffer(bytes(r.opaque), dtype=np.float64)[:rot // 2] * (2 * math.pi)
    want = ok.rope_thetas(rot, 500000.0, scaling, 8.0, 4096, 1.0, 4.0)
    assert np.allclose(got, want, rtol=1e-14, atol=0)


def test_rope_refusals():
    r = att.rope_encode(64)
    x = heads()
    refused(lambda: att.rope_apply(r, x, x, 0), "ERR_NULL")
    refused(lambda: att.rope_apply(r, heads(dtype="u16"), heads(dtype="u16"), BASE), "ERR_DTYPE")
    refused(lambda: att.rope_apply(r, heads(dtype="f64"), heads(dtype="f64"), BASE), "ERR_DTYPE")
    refused(lambda: att.rope_apply(r, x, heads(dtype="f16"), BASE), "ERR_UNSUPPORTED")
    refused(lambda: att.rope_apply(r, x, heads(n=9), BASE), "ERR_UNSUPPORTED")
    refused(lambda: att.rope_apply(r, heads(dim=48), heads(dim=48), BASE), "ERR_UNSUPPORTED")
    refused(lambda: att.rope_apply(r, heads(dim=264), heads(dim=264), BASE), "ERR_UNSUPPORTED")
    refused(lambda: att.rope_apply(r, pool(), pool(), BASE), "ERR_RANK")
    refused(lambda: att.rope_apply(att.rope_t(), x, x, BASE), "ERR_UNSUPPORTED")      # a plan that was not encoded
    strided = heads(estride=(1, 2, 1))
    refused(lambda: att.rope_apply(r, strided, strided, BASE), "ERR_UNSUPPORTED")
    # in place takes the same strides
    wide = att.tmap_encode("bf16", 3, BASE, (128, 8, 16), (512, 4096), (8, 1, 1))
    refused(lambda: att.rope_apply(r, x, wide, BASE), "ERR_UNSUPPORTED")


def test_append_refusals():
    r, q, k, p, t = att.rope_encode(64), heads(n=8), heads(n=2), pool(), table()

    def call(r=r, q=q, qo=q, k=k, v=k, kp=p, vp=p, pt=t, rows=BASE, at=BASE, pos=BASE):
        return lambda: att.rope_append(r, q, qo, k, v, kp, vp, pt, rows, at, pos)

    for c in (call(rows=0), call(at=0), call(pos=0), call(qo=None), call(q=None), call(pt=table(t=0)),
              call(k=None), call(vp=None)):
        refused(c, "ERR_NULL")
    for c in (call(k=heads(n=3)), call(v=heads(n=2, tokens=15)), call(kp=pool(slots=8)), call(vp=pool(dim=64)),
              call(kp=pool(pages=63)), call(pt=table(slots=8)), call(pt=table(pages=65)), call(q=heads(n=8, dim=64)),
              call(q=heads(tokens=17), qo=heads(tokens=17)), call(kp=pool(dtype="f16")),
              call(pt=table(pitch=7)), call(r=att.rope_encode(130))):
        refused(c, "ERR_UNSUPPORTED")
    refused(call(k=heads(n=2, dtype="u16"), v=heads(n=2, dtype="u16")), "ERR_DTYPE")


def test_page_refusals():
    p, t = pool(), table()
    ws = att.page_workspace(t, 4)
    assert ws > 0
    att.page_copy(p, 0, 0, 0)                       # nothing to do
    att.page_free(t, 0, 0)
    att.page_extend(t, 0, 0, 0, 0, 0)
    att.page_fork(t, p, 0, 0, 0, 0, 0)
    refused(lambda: att.page_copy(p, 0, BASE, 1), "ERR_NULL")
    refused(lambda: att.page_copy([], BASE, BASE, 1), "ERR_UNSUPPORTED")
    refused(lambda: att.page_copy([p, pool(slots=8)], BASE, BASE, 1), "ERR_UNSUPPORTED")
    refused(lambda: att.page_copy([p, pool(dtype="f16")], BASE, BASE, 1), "ERR_UNSUPPORTED")
    refused(lambda: att.page_copy([p] * 257, BASE, BASE, 1), "ERR_UNSUPPORTED")
    refused(lambda: att.page_copy(heads(), BASE, BASE, 1), "ERR_RANK")
    refused(lambda: att.page_free(t, 0, 1), "ERR_NULL")
    for bad in (table(rows=0), table(row_pages=0, pitch=1), table(pages=0), table(slots=0), table(pitch=7),
                table(row_pages=1 << 21), table(slots=1 << 20, row_pages=1 << 12)):
        refused(lambda: att.page_free(bad, BASE, 1), "ERR_UNSUPPORTED")
    refused(lambda: att.page_free(table(refs=0), BASE, 1), "ERR_NULL")
    refused(lambda: att.page_extend(t, BASE, BASE, 4, BASE, BASE, ws_bytes=16), "ERR_UNSUPPORTED")
    refused(lambda: att.page_extend(t, BASE, BASE, 4, BASE, BASE + 8, ws_bytes=1 << 20), "ERR_ALIGN")
    refused(lambda: att.page_extend(t, BASE, BASE, 4, 0, BASE, ws_bytes=1 << 20), "ERR_NULL")
    refused(lambda: att.page_extend(t, BASE, BASE, 4, BASE, 0, ws_bytes=1 << 20), "ERR_NULL")
    refused(lambda: att.page_fork(t, pool(slots=8), BASE, BASE, 4, BASE, BASE, ws_bytes=1 << 20), "ERR_UNSUPPORTED")
    refused(lambda: att.page_fork(t, p, BASE, 0, 4, BASE, BASE, ws_bytes=1 << 20), "ERR_NULL")
    refused(lambda: att.page_compact(t, table(rows=7), p, 0, BASE, ws_bytes=1 << 20), "ERR_UNSUPPORTED")
    refused(lambda: att.page_compact(t, table(pitch=9), p, 0, BASE, ws_bytes=1 << 20), "ERR_UNSUPPORTED")
    refused(lambda: att.page_compact(t, t, pool(pages=32), 0, BASE, ws_bytes=1 << 20), "ERR_UNSUPPORTED")
    refused(lambda: att.page_compact(t, t, p, 0, BASE, ws_bytes=16), "ERR_UNSUPPORTED")


def test_page_table_of_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros((4, 6), dtype=torch.int32)
    pt = att.page_table(t[:, :5], torch.zeros(4, dtype=torch.int32), None, 9, 16)
    assert (pt.rows, pt.row_pages, pt.pitch, pt.pages, pt.slots, pt.d_refs) == (4, 5, 6, 9, 16, None)
    with pytest.raises(ValueError):
        att.page_table(t.t(), None, None, 9, 16)
    with pytest.raises(TypeError):
        att.page_table(t.long(), None, None, 9, 16)


def test_attention_refusals():
    q, p, t = queries(), pool(), table()
    ws = att.attn_workspace(q, p, 100, 64)
    assert ws > 0

    def call(q=q, k=p, v=p, pt=t, prow=0, plen=100, o=q, scale=0.1, d_ws=BASE, n=ws):
        return lambda: att.attn_shared_prefix(q, k, v, pt, prow, plen, 0, 64, scale, o, 0, d_ws, 0, n)

    for c in (call(q=None), call(d_ws=0), call(pt=table(lens=0)), call(pt=table(t=0))):
        refused(c, "ERR_NULL")
    for c in (call(q=queries(n=7), o=queries(n=7)), call(v=pool(n=4)), call(o=queries(batch=5)), call(plen=129),
              call(prow=8), call(pt=table(slots=8)), call(scale=float("nan")), call(n=ws - 1),
              call(k=pool(dtype="f16")), call(q=queries(dim=64), o=queries(dim=64)),
              call(q=queries(dim=264), o=queries(dim=264), k=pool(dim=264), v=pool(dim=264))):
        refused(c, "ERR_UNSUPPORTED")
    refused(call(d_ws=BASE + 8), "ERR_ALIGN")
    refused(call(q=heads()), "ERR_RANK")
    refused(call(q=att.tmap_encode("f32", 4, BASE, (128, 8, 1, 4), (512, 4096, 4096), (4, 1, 1, 1))), "ERR_DTYPE")
    assert att.attn_workspace(heads(), p, 0, 0) == 0


# ---- the oracle, by hand ---------------------------------------------------------

def test_oracle_rope_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y, _ = ok.rope(x, [1], [math.pi / 2, math.pi], "half", 2.0)
    assert np.allclose(y, [[[-6.0, -4.0, 2.0, -8.0, 5.0]]])
    y, _ = ok.rope(x, [1], [math.pi / 2, math.pi], "interleaved")
    assert np.allclose(y, [[[-2.0, 1.0, -3.0, -4.0, 5.0]]])
    z, _ = ok.rope(y, [1], [math.pi / 2, math.pi], "interleaved", inverse=True)
    assert np.allclose(z, x)


def test_oracle_pages_by_hand():
    table = np.full((4, 3), -1, dtype=np.int32)
    table[0, :2] = [5, 2]
    p = ok.Pages(table, np.array([6, 0, 0, 0]), np.array([0, 0, 1, 0, 0, 1, 0]), 4, [np.arange(7)])
    assert p.fork([0, 0], [2, 3]) == [1, 1]
    assert p.table.tolist() == [[5, 2, -1], [-1, -1, -1], [5, 0, -1], [5, 1, -1]]
    assert p.refs.tolist() == [1, 1, 1, 0, 0, 3, 0] and p.pools[0].tolist() == [2, 2, 2, 3, 4, 5, 6]
    assert p.extend([2, 3, 0], [2, 3, 7]) == [1, 1, 0]        # the third row is too short for 13 tokens
    assert p.table.tolist() == [[5, 2, -1], [-1, -1, -1], [5, 0, -1], [5, 1, 3]]
    p.free([0, 2, 2])
    assert p.refs.tolist() == [0, 1, 0, 1, 0, 1, 0] and p.lens.tolist() == [0, 0, 0, 9]
    assert p.compact() == 3
    assert p.table[3].tolist() == [2, 1, 0] and p.refs.tolist() == [1, 1, 1, 0, 0, 0, 0]
    assert p.pools[0].tolist()[:3] == [3, 2, 5]


def test_oracle_attention_empty_and_uniform():
    q = np.zeros((2, 1, 2, 8))
    pool_ = np.arange(3 * 2 * 1 * 8, dtype=np.float64).reshape(3, 2, 1, 8)
    o, lse, *_ = ok.attention(q, pool_, pool_, np.array([[0, 1], [2, -1]]), np.array([3, 0]), 2, 0, 0, None, 1.0)
    assert np.allclose(o[0, 0, 0], pool_.reshape(6, 8)[[0, 1, 2]].mean(0)) and np.isclose(lse[0, 0, 0], math.log(3))
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
