"""The paged cache's calls in the forms that only larger work takes: prefix
tiles shared by four waves at every padded head size, outputs that stream past
the caches, more pools than the small launches carry.  Tolerances as in
test_gpu_kvcache.py."""
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


# ---- shared prefix tiles: rows above 64, kv * rows * prefix above 10^7 ----------------

SHARED = [  # as ATTN in test_gpu_kvcache.py; rows not whole blocks of 128, prefixes not whole tiles of 64
    ("bf16", 70, 1, 16, 16, 128, 16, 9001, [(3 * i) % 40 for i in range(70)], False, 0),
    ("f16", 45, 3, 32, 8, 128, 48, 2333, [(5 * i) % 70 for i in range(45)], True, 8),
    ("bf16", 45, 3, 32, 8, 104, 7, 2333, [i % 5 for i in range(45)], False, 0),
    ("bf16", 40, 2, 12, 4, 192, 7, 10501, [(7 * i) % 50 for i in range(40)], True, 0),
    ("f16", 70, 1, 16, 16, 192, 16, 9001, [i % 3 for i in range(70)], False, 8),
    ("f16", 70, 1, 16, 16, 176, 16, 9001, [i % 3 for i in range(70)], False, 0),
    ("f16", 65, 1, 32, 32, 256, 32, 4999, [(3 * i) % 35 for i in range(65)], False, 0),
    ("bf16", 13, 5, 96, 48, 96, 16, 1701, [i for i in range(13)], False, 0),
    ("bf16", 67, 1, 64, 64, 24, 100, 2401, [i % 4 for i in range(67)], True, 0),
]


@pytest.mark.parametrize("hint", [0, 100])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_tiles(case, hint, monkeypatch):
    c = SHARED[case]
    dtype, batch, q_len, heads, kv, dim, slots, prefix = c[:8]
    rows_all = batch * q_len * heads // kv
    assert rows_all > 64 and kv * rows_all * prefix > 10 ** 7 and rows_all % 128 and prefix % 64
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(600 + case))
    got, lse = base.attn_run(q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype, hint)
    monkeypatch.setattr(ok, "attention", ok.attention_by_head)
    base.attn_check(got, lse, q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype)


@pytest.mark.parametrize("dtype, dim", [("bf16", 128), ("f16", 192), ("bf16", 256), ("f16", 96)])
def test_shared_tiles_keep_what_is_not_finite_apart(dtype, dim):
    """80 rows over 500 heads: a NaN in one query, in one key, an infinity in
    one value and pages that are not there reach those who see them, only."""
    batch, kv, prefix = 80, 500, 300
    c = (dtype, batch, 1, kv, kv, dim, 16, prefix, [5] * batch, False, 0)
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(61))

    def run(t=table):
        return base.attn_run(q, kp, vp, t, lens, rows, 16, prefix, dim ** -0.5, dtype)

    clean, lse = run()
    q[7, 0, 3, dim - 1] = math.nan
    got, lse2 = run()
    assert np.isnan(got[7, 0, 3]).all() and np.isnan(lse2[7, 0, 3])
    got[7, 0, 3], lse2[7, 0, 3] = clean[7, 0, 3], lse[7, 0, 3]
    assert np.array_equal(got, clean) and np.array_equal(lse2, lse)
    q[7, 0, 3, dim - 1] = 0.5
    clean, lse = run()
    vp[int(table[1][7]), 3, 4, 11] = math.inf
    got, lse2 = run()
    assert np.isposinf(got[:, 0, 4, 11]).all()
    got[:, 0, 4, 11] = clean[:, 0, 4, 11]
    assert np.array_equal(got, clean) and np.array_equal(lse2, lse)
    vp[int(table[1][7]), 3, 4, 11] = 0.25
    kp[int(table[1][2]), 9, 6, 0] = math.nan
    clean, lse = run()
    assert np.isnan(clean[:, 0, 6]).all() and np.isnan(lse[:, 0, 6]).all()
    clean[:, 0, 6] = lse[:, 0, 6] = 0
    assert np.isfinite(clean).all() and np.isfinite(lse).all()
    kp[int(table[1][2]), 9, 6, 0] = 0.25
    # a page that is not there against values and keys of the same page that nobody sees: the same results
    bad = table.copy()
    bad[1, 11] = kp.shape[0]
    clean, lse = run(bad)
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    kp[int(table[1][11])], vp[int(table[1][11])] = math.nan, math.inf
    got, lse2 = run(bad)
    with pytest.raises(att.TmapError):
        att.tile_device_status(stream())
    assert np.isfinite(clean).all() and np.array_equal(got, clean) and np.array_equal(lse2, lse)


# ---- many queries of one sequence: several blocks of 32, several placements of keys ---

PROMPT = [
    ("bf16", 1, 700, 4, 2, 128, 16, 0, [700], False, 0),
    ("f16", 2, 333, 6, 2, 64, 48, 150, [333, 900], True, 0),
    ("bf16", 3, 129, 3, 1, 192, 7, 1000, [5, 129, 600], False, 8),
    ("f16", 1, 513, 2, 2, 256, 16, 70, [1030], False, 0),
]


@pytest.mark.parametrize("hint", [0, 600])
@pytest.mark.parametrize("case", range(len(PROMPT)))
def test_prompts(case, hint, monkeypatch):
    c = PROMPT[case]
    dtype, dim, slots, prefix = c[0], c[5], c[6], c[7]
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(700 + case))
    got, lse = base.attn_run(q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype, hint)
    monkeypatch.setattr(ok, "attention", ok.attention_by_head)
    base.attn_check(got, lse, q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype)


@pytest.mark.parametrize("case", range(len(PROMPT)))
def test_prompts_do_not_see_what_follows(case):
    """NaN and infinities from one token of each sequence on reach the queries
    from that token on, no other."""
    c = PROMPT[case]
    dtype, batch, q_len, dim, slots, prefix, length = c[0], c[1], c[2], c[5], c[6], c[7], c[8]
    q, kp, vp, table, lens, rows = base.attn_setup(c, base.gen(750 + case))
    clean, lse = base.attn_run(q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype)
    first = [max(0, n - 77) for n in length]                 # the first token that is not finite
    for b, t0 in enumerate(first):
        for t in range(t0, length[b]):
            page = int(table[rows[b]][t // slots])
            kp[page, t % slots] = math.nan if t % 2 else math.inf
            vp[page, t % slots] = math.inf if t % 3 else math.nan
    got, lse2 = base.attn_run(q, kp, vp, table, lens, rows, slots, prefix, dim ** -0.5, dtype)
    for b in range(batch):
        j = first[b] - (length[b] - q_len)                   # the query whose own token that is
        assert np.array_equal(got[b, :j], clean[b, :j]) and np.array_equal(lse2[b, :j], lse[b, :j])
        assert not np.isfinite(got[b, j:]).any()


# ---- outputs above 32 MiB --------------------------------------------------------------

def streamed(x):
    return x.numel() * x.element_size() > 32 << 20


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dtype, tokens, heads, dim, rot, layout", [
    ("bf16", 8191, 17, 128, 128, "half"), ("f16", 4099, 33, 136, 96, "half"), ("bf16", 4099, 33, 128, 42, "half"),
    ("f16", 8191, 17, 128, 128, "interleaved"), ("f32", 8195, 9, 116, 70, "interleaved"),
    ("f32", 4097, 10, 256, 256, "half"), ("f32", 70001, 1, 120, 6, "half"), ("bf16", 8191, 18, 124, 32, "interleaved")])
def test_rope_streams(dtype, tokens, heads, dim, rot, layout, inverse):
    """The whole output against calls small enough not to stream, bit by bit,
    and a sample of its tokens against the oracle."""
    g = base.gen(tokens)
    _, x = base.padded((tokens, heads, dim), dtype, 0, g)
    _, y = base.padded((tokens, heads, dim), dtype, 8, g)
    assert streamed(x)
    pos = torch.randint(-5000, 1 << 20, (tokens,), generator=g).to(torch.int32)
    p = pos.cuda()
    plan = att.rope_encode(rot, layout, 10000.0, "ramp", 4.0, 4096)
    att.rope_apply(plan, base.tensor_map(x, dtype), base.tensor_map(y, dtype), p, inverse, stream())
    for a in range(0, tokens, 1500):
        n = min(tokens, a + 1500) - a
        part = torch.zeros((n, heads, -(-dim // 8) * 8), dtype=x.dtype, device="cuda")[..., :dim]
        assert not streamed(part)
        att.rope_apply(plan, base.tensor_map(x[a:a + 1500], dtype), base.tensor_map(part, dtype), p[a:a + 1500], inverse,
                       stream())
        assert torch.equal(part, y[a:a + 1500])
    some = sorted({0, 1, tokens - 2, tokens - 1, *range(0, tokens, tokens // 40)})
    want, size = ok.rope(base.f64(x[some]), pos[some].numpy(),
                         ok.rope_thetas(rot, 10000.0, "ramp", 4.0, 4096), layout, 1.0, inverse)
    limit = base.rope_limit(want, size, dtype) + size * 2.0 ** (20 - 52)
    assert (np.abs(base.f64(y[some]) - want) <= limit).all()
    # in place
    att.rope_apply(plan, base.tensor_map(x, dtype), base.tensor_map(x, dtype), p, inverse, stream())
    assert torch.equal(x, y)


@pytest.mark.parametrize("dtype, tokens, heads, kv, dim, rot, layout", [
    ("bf16", 4099, 18, 8, 128, 128, "half"), ("f16", 4099, 18, 8, 128, 42, "half"), ("f32", 4099, 5, 5, 144, 64, "half"),
    ("bf16", 2049, 33, 17, 128, 64, "interleaved"), ("f16", 4099, 0, 18, 120, 120, "half")])
def test_append_streams(dtype, tokens, heads, kv, dim, rot, layout):
    g = base.gen(heads)
    slots, rows = 48, 3
    row_pages = -(-tokens // slots)
    pages = rows * row_pages
    table = torch.randperm(pages, generator=g).view(rows, row_pages).to(torch.int32).cuda()
    pt = att.page_table(table, None, None, pages, slots)
    q, k, v = (torch.randn((tokens, n or 1, dim), generator=g).to(base.TORCH[dtype]).cuda() for n in (heads, kv, kv))
    assert (heads + 2 * kv) * tokens * dim * q.element_size() > 32 << 20
    pools = [torch.zeros((pages, slots, kv, dim), dtype=base.TORCH[dtype], device="cuda") for _ in range(4)]
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    row = torch.randint(0, rows, (tokens,), generator=g).to(torch.int32).cuda()
    row[5] = -1
    at = torch.randperm(row_pages * slots, generator=g)[:tokens].to(torch.int32).cuda()
    plan = att.rope_encode(rot, layout)

    def append(a, b, o, kp, vp):
        m = [base.tensor_map(t[a:b], dtype) for t in (q, o, k, v)]
        att.rope_append(plan, *(m if heads else [None, None, *m[2:]]), base.pool_map(kp, dtype), base.pool_map(vp, dtype), pt,
                        row[a:b], at[a:b], at[a:b], stream())

    append(0, tokens, out, pools[0], pools[1])
    for a in range(0, tokens, 999):
        append(a, min(tokens, a + 999), want, pools[2], pools[3])
    assert torch.equal(out, want) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    keep = row >= 0
    page = table[row[keep].long(), (at[keep] // slots).long()].long()
    assert torch.equal(pools[1][page, (at[keep] % slots).long()], v[keep])


# ---- more than 16 pools ------------------------------------------------------------------

@pytest.mark.parametrize("pages, npool", [(60, 16), (60, 17), (60, 256), (9000, 16), (9000, 17), (9000, 100)])
def test_many_pools(pages, npool):
    """Copy, fork, and compaction into the same table and into another, of few
    pages (one launch into another table) and many (two)."""
    slots, rows, row_pages, dim = 3, 7, 6, 8
    rng = np.random.default_rng(npool)
    whole = torch.randint(-999, 999, (npool, pages, slots, 2, dim), generator=base.gen(npool)).to(torch.int16).cuda()
    pools = list(whole)
    maps = att.tmap_array([base.pool_map(p, "u16") for p in pools])
    used = rng.permutation(pages)[:20]
    table = np.full((rows, row_pages), -1, dtype=np.int32)
    table[0, :5], table[1, :6], table[2, :3], table[3, :6] = np.split(used, [5, 11, 14])
    lens = np.array([14, 18, 7, 16, 0, 0, 0], dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    refs[used] = 1
    want = ok.Pages(table, lens, refs, slots, [p.cpu().numpy() for p in pools])
    d_table, d_lens, d_refs = base.ints(table), base.ints(lens), base.ints(refs)
    pt = att.page_table(d_table, d_lens, d_refs, pages, slots)
    ws = torch.empty(att.page_workspace(pt, rows), dtype=torch.uint8, device="cuda")
    flag = base.ints([9] * 3)
    att.page_fork(pt, maps, base.ints([0, 2, 1]), base.ints([4, 6, 5]), 3, flag, ws, stream())
    assert flag.tolist() == want.fork([0, 2, 1], [4, 6, 5])
    base.same(d_table, d_lens, d_refs, pools, want)
    src, dst = int(used[3]), int(next(p for p in range(pages) if want.refs[p] == 0))
    att.page_copy(maps, base.ints([src, -1]), base.ints([dst, 0]), 2, stream())
    for p in want.pools:
        p[dst] = p[src]
    base.same(d_table, d_lens, d_refs, pools, want)
    for here in (False, True):
        gone = [1] if here else [0, 6]
        att.page_free(pt, base.ints(gone), len(gone), stream())
        want.free(gone)
        used_now = base.ints([-1])
        if here:
            att.page_compact(pt, pt, maps, used_now, ws, stream())
        else:
            t2, r2 = torch.full_like(d_table, -3), torch.full_like(d_refs, -3)
            att.page_compact(pt, att.page_table(t2, d_lens, r2, pages, slots), maps, used_now, ws, stream())
            d_table.copy_(t2)
            d_refs.copy_(r2)
        assert used_now.item() == want.compact()
        base.same(d_table, d_lens, d_refs, pools, want)
