"""Host side of the paged cache's calls at the limits of their arguments (no
GPU): refusals come before any HIP call."""
import pytest

import async_tensor_tile_amd as att

from test_kvcache_host import BASE, heads, pool, queries, refused, table  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38, float("inf")])
def test_scale_beyond_powers_of_two(scale):
    """Scores are kept in powers of two, so scale * log2(e) has to be finite."""
    q, p = queries(), pool()
    ws = att.attn_workspace(q, p, 100, 64)
    refused(lambda: att.attn_shared_prefix(q, p, p, table(), 0, 100, 0, 64, scale, q, 0, BASE, 0, ws),
            "ERR_UNSUPPORTED")


@pytest.mark.parametrize("args", [dict(rot_dim=64, magnitude=1e39),                       # infinite in fp32
                                  dict(rot_dim=64, scaling="base", base=1e300, factor=1e9),  # so is the scaled base
                                  dict(rot_dim=64, scaling="base", base=1e-300, factor=1e-30),
                                  dict(rot_dim=64, scaling="linear", factor=1e-308),
                                  dict(rot_dim=64, scaling="ramp", factor=1e-308, original_len=64),
                                  dict(rot_dim=256, base=1e-307)])
def test_rope_plans_that_cannot_be_held(args):
    refused(lambda: att.rope_encode(**args), "ERR_UNSUPPORTED")


@pytest.mark.parametrize("args", [dict(rot_dim=64, magnitude=3e38), dict(rot_dim=64, base=1e300),
                                  dict(rot_dim=64, base=1e-290), dict(rot_dim=2, scaling="base", factor=1e300)])
def test_rope_plans_at_the_limits(args):
    att.rope_encode(**args)


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) - 1])
def test_entries_that_32_bits_cannot_step_through(n):
    refused(lambda: att.page_extend(table(), BASE, BASE, n, BASE, BASE, ws_bytes=1 << 40), "ERR_UNSUPPORTED")
    refused(lambda: att.page_fork(table(), pool(), BASE, BASE, n, BASE, BASE, ws_bytes=1 << 40), "ERR_UNSUPPORTED")


def test_attention_beyond_one_launch():
    """2^24 - 1 workgroups of 256 threads: one for each sequence and head here."""
    p = pool(n=512)
    assert att.attn_workspace(queries(n=512, batch=32767), p, 0, 0) > 0
    for prefix in (0, 100):
        q = queries(n=512, batch=32768)
        assert att.attn_workspace(q, p, prefix, 0) == 0
        refused(lambda: att.attn_shared_prefix(q, p, p, table(rows=40000), 0, prefix, 0, 0, 0.1, q, 0, BASE, 0, 1 << 40),
                "ERR_UNSUPPORTED")
    # many queries of one sequence
    q = queries(n=64, q_len=65535, batch=128)
    assert att.attn_workspace(q, pool(n=4), 0, 0) == 0


def u8_pool(dims, strides):
    return att.tmap_encode("u8", 4, BASE, dims, strides, (16, 1, 1, 1))


def test_pages_above_256_mib():
    """n == 0 checks the pools alone.  Bytes of a page that wrap 64 bits count too."""
    k = 1 << 14
    att.page_copy(u8_pool((k, k, 1, 2), (k, k * k, k * k)), BASE, BASE, 0)
    big = [u8_pool((k, k + 1, 1, 2), (k, k * (k + 1), k * (k + 1))),
           u8_pool((k, 1, k + 1, 2), (k, k, k * (k + 1))),
           u8_pool((1, k, k // 4 + 1, 2), (16, 16 * k, 16 * k * k)),                  # rows of one byte, 16 each
           u8_pool((1 << 32, 1 << 32, 1, 2), (1 << 32, 1 << 39, 1 << 39)),            # 2^64 bytes in a packed row
           u8_pool((1 << 20, 1 << 32, 1 << 32, 2), (1 << 24, 1 << 39, 1 << 39))]      # 2^84, rows apart
    for p in big:
        refused(lambda: att.page_copy(p, BASE, BASE, 0), "ERR_UNSUPPORTED")


def test_tensors_of_other_types_and_strides_are_refused():
    """torch's own integers are int64: read as int32, every other value is 0."""
    torch = pytest.importorskip("torch")
    wrong = [(torch.zeros(16, dtype=torch.int64), TypeError), (torch.zeros(16), TypeError),
             (torch.zeros(16, dtype=torch.int16), TypeError), (torch.zeros(32, dtype=torch.int32)[::2], ValueError)]
    good = torch.zeros(16, dtype=torch.int32)
    r, x, k, p, t, q = att.rope_encode(64), heads(), heads(n=2), pool(), table(), queries()
    ws = torch.empty(att.page_workspace(t, 4), dtype=torch.uint8)
    calls = {
        "d_pos": lambda a: att.rope_apply(r, x, x, a),
        "d_rows": lambda a: att.rope_append(r, None, None, k, k, p, p, t, a, good, good),
        "d_at": lambda a: att.rope_append(r, None, None, k, k, p, p, t, good, a, good),
        "d_pos ": lambda a: att.rope_append(r, None, None, k, k, p, p, t, good, good, a),
        "d_src": lambda a: att.page_copy(p, a, good, 4),
        "d_dst": lambda a: att.page_copy(p, good, a, 4),
        "d_rows ": lambda a: att.page_extend(t, a, good, 4, good, ws),
        "d_add": lambda a: att.page_extend(t, good, a, 4, good, ws),
        "d_ok": lambda a: att.page_extend(t, good, good, 4, a, ws),
        "d_src ": lambda a: att.page_fork(t, p, a, good, 4, good, ws),
        "d_dst ": lambda a: att.page_fork(t, p, good, a, 4, good, ws),
        "d_ok ": lambda a: att.page_fork(t, p, good, good, 4, a, ws),
        "d_rows  ": lambda a: att.page_free(t, a, 4),
        "d_used": lambda a: att.page_compact(t, t, p, a, ws),
        "d_rows   ": lambda a: att.attn_shared_prefix(q, p, p, t, 0, 0, a, 0, 0.1, q, 0, ws),
    }
    for name, call in calls.items():
        for a, error in wrong:
            with pytest.raises(error, match=name.strip()):
                call(a)
    for a in (torch.zeros(16, dtype=torch.float64), torch.zeros(16, dtype=torch.int32), torch.zeros(32)[::2]):
        with pytest.raises(TypeError, match="d_lse"):
            att.attn_shared_prefix(q, p, p, t, 0, 0, 0, 0, 0.1, q, a, ws)


def test_page_tables_of_short_tensors_are_refused():
    torch = pytest.importorskip("torch")

    def new(n):
        return torch.zeros(n, dtype=torch.int32)

    att.page_table(new((4, 5)), new(4), new(9), 9, 16)
    att.page_table(new((4, 5)), new(6), new(12), 9, 16)
    for lens, refs in ((new(3), new(9)), (new(4), new(8)), (new(8)[::2], new(9)), (new(4), new(18)[::2])):
        with pytest.raises(ValueError):
            att.page_table(new((4, 5)), lens, refs, 9, 16)


def test_page_tables_whose_rows_share_memory_are_refused():
    """An expanded table has a stride of 0, which is not a pitch."""
    torch = pytest.importorskip("torch")
    t = torch.zeros((1, 5), dtype=torch.int32)
    lens, refs = torch.zeros(4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    assert att.page_table(t, lens, refs, 9, 16).pitch == 5
    with pytest.raises(ValueError):
        att.page_table(t.expand(4, 5), lens, refs, 9, 16)
    with pytest.raises(ValueError):
        att.page_table(torch.zeros(8, dtype=torch.int32).as_strided((4, 5), (1, 1)), lens, refs, 9, 16)
