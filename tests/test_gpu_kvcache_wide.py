"""The paged cache's calls with more work than one launch holds (2^32 - 1 threads
along a dimension), against the same calls piece by piece."""
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402

import test_gpu_kvcache as base  # noqa: E402
from gpu_util import require_native, stream  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


# ---- rotary positions: two tokens of 256 threads --------------------------------------

TOKENS = (1 << 25) + 1029


def pieces():
    """Cuts that do not meet those between launches."""
    at = [0, 1 << 23, (1 << 24) + 7, (1 << 25) - 1000, TOKENS]
    return list(zip(at, at[1:]))


@pytest.mark.parametrize("layout, rot", [("half", 6), ("interleaved", 8)])
def test_rope_of_many_tokens(layout, rot):
    x = torch.randn((TOKENS, 1, 8), device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (TOKENS,), dtype=torch.int32, device="cuda")
    y, want = torch.empty_like(x), torch.empty_like(x)
    plan = att.rope_encode(rot, layout)
    att.rope_apply(plan, base.tensor_map(x, "bf16"), base.tensor_map(y, "bf16"), pos, False, stream())
    for a, b in pieces():
        att.rope_apply(plan, base.tensor_map(x[a:b], "bf16"), base.tensor_map(want[a:b], "bf16"), pos[a:b], False,
                       stream())
    assert torch.equal(y, want)


def test_append_of_many_tokens():
    slots = 4096
    pages = -(-TOKENS // slots)
    q, k, v = (torch.randn((TOKENS, 1, 8), device="cuda").to(torch.float16) for _ in "qkv")
    pools = [torch.zeros((pages, slots, 1, 8), dtype=torch.float16, device="cuda") for _ in range(4)]
    out, want = torch.empty_like(q), torch.empty_like(q)
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None].contiguous()
    pt = att.page_table(table, None, None, pages, slots)
    rows = torch.zeros(TOKENS, dtype=torch.int32, device="cuda")
    at = torch.arange(TOKENS, dtype=torch.int32, device="cuda")
    plan = att.rope_encode(8)

    def append(a, b, o, kp, vp):
        att.rope_append(plan, *(base.tensor_map(t[a:b], "f16") for t in (q, o, k, v)), base.pool_map(kp, "f16"),
                        base.pool_map(vp, "f16"), pt, rows[a:b], at[a:b], at[a:b], stream())

    append(0, TOKENS, out, pools[0], pools[1])
    for a, b in pieces():
        append(a, b, want, pools[2], pools[3])
    att.tile_device_status(stream())
    assert torch.equal(out, want) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert torch.equal(pools[1][table[0].long()].view(-1, 8)[:TOKENS], v[:, 0])


# ---- pages: an entry of 256 threads -----------------------------------------------------

ENTRIES = (1 << 24) + 100


def test_page_copy_of_many_entries():
    """Nearly all skipped; those on either side of the cut are copied."""
    pools = torch.randint(-999, 999, (64, 4, 1, 8), device="cuda").to(torch.int16)
    src = torch.full((ENTRIES,), -1, dtype=torch.int32, device="cuda")
    dst = src.clone()
    want = pools.clone()
    for k, i in enumerate([0, 5, (1 << 24) - 3, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, ENTRIES - 1]):
        src[i], dst[i] = k, 32 + k
        want[32 + k] = pools[k]
    att.page_copy(base.pool_map(pools, "u16"), src, dst, ENTRIES, stream())
    assert torch.equal(pools, want)


def test_fork_and_free_of_many_rows():
    """A finished page shared by 2^24 and more rows, and given back by all."""
    rows = ENTRIES + 1
    table = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = base.ints([0, 0, 1])
    table[0, 0], lens[0] = 2, 4
    pt = att.page_table(table, lens, refs, 3, 4)
    dst = torch.arange(rows - 1, 0, -1, dtype=torch.int32, device="cuda")
    src = torch.zeros_like(dst)
    flag = torch.empty_like(dst)
    ws = torch.empty(att.page_workspace(pt, ENTRIES), dtype=torch.uint8, device="cuda")
    att.page_fork(pt, None, src, dst, ENTRIES, flag, ws, stream())
    assert (flag == 1).all() and (table == 2).all() and (lens == 4).all() and refs.tolist() == [0, 0, rows]
    att.page_free(pt, dst, ENTRIES, stream())
    assert (table[1:] == -1).all() and (lens[1:] == 0).all() and refs.tolist() == [0, 0, 1]
    att.tile_device_status(stream())


def test_fork_of_many_large_pages():
    """256 pools with pages of 4 MiB: more parts of a page than a grid is high."""
    slots, npool = 512, 256
    pools = torch.empty((npool, 2, slots, 8, 1024), dtype=torch.uint8, device="cuda")
    pools[:, 1].random_(0, 255)
    pools[:, 0] = 0
    maps = att.tmap_array([base.pool_map(p, "u8") for p in pools])
    table, lens, refs = base.ints([[1], [-1]]), base.ints([5, 0]), base.ints([0, 1])
    pt = att.page_table(table, lens, refs, 2, slots)
    ws = torch.empty(att.page_workspace(pt, 1), dtype=torch.uint8, device="cuda")
    flag = base.ints([9])
    att.page_fork(pt, maps, base.ints([0]), base.ints([1]), 1, flag, ws, stream())
    assert flag.tolist() == [1] and table.tolist() == [[1], [0]] and refs.tolist() == [1, 1]
    assert torch.equal(pools[:, 0], pools[:, 1])
