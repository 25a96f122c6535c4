"""GPU parity of the paged cache's calls against the 64-bit oracle.

Tolerances count roundings.  One rounding to a type is off by at most half a
step (bf16 2^-8, fp16 2^-11, fp32 2^-24, relative).  Rotation: cosine and sine
carry at most 2^-21 (angle in fp32 turns, the function, the magnitude), which
scales with |a| + |b| of the pair; then one rounding to the type.  Attention: a
score is a sum of dim products in fp32, so it is off by at most (dim + 8) *
2^-24 times the sum of their absolute values; that shifts a weight by as much
again, relatively, and the exponential adds 2^-21.  Each weight is rounded to
the type for the product with the values, n of those are added in fp32, and
the quotient is rounded to the type."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "u8": torch.uint8, "u16": torch.int16}


def setup_module(module):
    require_native()


def f64(t):
    return t.detach().double().cpu().numpy()


def tensor_map(t, dtype):
    """Map of a torch tensor, whatever its strides (innermost contiguous)."""
    e = t.element_size()
    return att.tmap_encode(dtype, t.dim(), t.data_ptr(), tuple(reversed(t.shape)),
                           tuple(s * e for s in reversed(t.stride()[:-1])), (16 // e,) + (1,) * (t.dim() - 1))


def padded(shape, dtype, gap, g, junk=float("nan")):
    """Random tensor whose rows are `gap` elements longer than its last
    dimension (rounded up to whole 16 bytes); the gap holds junk."""
    n = 16 // torch.empty(0, dtype=TORCH[dtype]).element_size()
    wide = -(-(shape[-1] + gap) // n) * n
    t = torch.full(shape[:-1] + (wide,), junk, dtype=torch.float32).to(TORCH[dtype]).cuda()
    v = t[..., :shape[-1]]
    v.copy_(torch.randn(shape, generator=g).to(TORCH[dtype]))
    return t, v


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---- rotary positions --------------------------------------------------------------

def rope_limit(want, size, dtype):
    return ok.half_step(dtype) * np.abs(want) + 2.0 ** -21 * size + (2.0 ** -25 if dtype == "f16" else 1e-37)


ROPE = [  # dtype, tokens, heads, dim, rot, layout, scaling, magnitude, gap
    ("bf16", 1, 1, 8, 2, "half", "none", 1.0, 0),
    ("bf16", 5, 3, 128, 128, "half", "none", 1.0, 0),
    ("bf16", 7, 2, 128, 64, "interleaved", "linear", 1.0, 8),
    ("f16", 33, 5, 96, 80, "half", "base", 1.25, 0),
    ("f16", 9, 4, 80, 42, "half", "none", 1.0, 8),
    ("f16", 4, 3, 100, 36, "interleaved", "ramp", 1.0, 4),
    ("f32", 6, 7, 64, 64, "half", "ramp", 0.5, 0),
    ("f32", 3, 2, 256, 254, "interleaved", "none", 1.0, 0),
    ("f32", 2, 2, 250, 6, "half", "none", 1.0, 2),
    ("bf16", 1025, 3, 72, 16, "half", "none", 1.0, 0),
    ("bf16", 1027, 9, 128, 128, "interleaved", "none", 1.0, 16),
    ("f16", 1, 40, 256, 256, "half", "none", 1.0, 0),
    ("f32", 1030, 2, 96, 96, "half", "base", 1.0, 0),
    ("bf16", 3, 2, 77, 30, "half", "none", 1.0, 3),
    ("bf16", 3, 2, 77, 32, "interleaved", "none", 1.0, 3),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope(case, inverse):
    dtype, tokens, n, dim, rot, layout, scaling, magnitude, gap = ROPE[case]
    g = gen(case)
    args = (10000.0, scaling, 4.0, 2048, 1.0, 32.0)
    _, x = padded((tokens, n, dim), dtype, gap, g)
    whole, y = padded((tokens, n, dim), dtype, gap + 8, g)
    before = whole.clone()
    pos = torch.randint(-5000, 1 << 20, (tokens,), generator=g).numpy()
    pos[0] = [0, 2 ** 31 - 1, -2 ** 31, 1][case % 4]
    plan = att.rope_encode(rot, layout, *args, magnitude)
    mx, my, p = tensor_map(x, dtype), tensor_map(y, dtype), ints(pos)
    att.rope_apply(plan, mx, my, p, inverse, stream())
    want, size = ok.rope(f64(x), pos, ok.rope_thetas(rot, *args), layout, magnitude, inverse)
    got = f64(y)
    limit = rope_limit(want, size, dtype)
    # fmod of the oracle's own product: position * theta is rounded to 53 bits
    limit += size * np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -52
    assert (np.abs(got - want) <= limit).all(), np.abs(got - want).max()
    assert np.array_equal(got[..., rot:], f64(x)[..., rot:])
    gap_now, gap_then = whole[..., dim:].cpu(), before[..., dim:].cpu()
    assert torch.equal(gap_now.view(torch.uint8), gap_then.view(torch.uint8))
    # in place
    att.rope_apply(plan, mx, mx, p, inverse, stream())
    assert torch.equal(x.cpu(), y.cpu())


def test_rope_gradient_against_differences():
    """The inverse call is the gradient: <g, R(x + h e) - R(x - h e)> / 2h."""
    g = gen(3)
    x = torch.randn((5, 2, 32), generator=g).cuda()
    up = torch.randn((5, 2, 32), generator=g).cuda()
    plan, pos = att.rope_encode(20, "half", 100.0, magnitude=1.5), ints([0, 1, 7, 100, 3000])

    def rotate(t, inverse=False):
        y = torch.empty_like(t)
        att.rope_apply(plan, tensor_map(t, "f32"), tensor_map(y, "f32"), pos, inverse, stream())
        return y

    grad = rotate(up, True)
    for i, j, k in [(0, 0, 0), (1, 1, 3), (2, 0, 13), (3, 1, 19), (4, 0, 20), (4, 1, 31)]:
        e = torch.zeros_like(x)
        e[i, j, k] = 0.5
        d = (rotate(x + e) - rotate(x - e)).double().mul(up.double()).sum().item()
        # each of the 64 elements of a token is off by 2^-21 of |a| + |b| (below 12) in either call
        assert abs(d - grad[i, j, k].item()) <= 2 * 64 * 12 * 2.0 ** -21 * up.abs().max().item()


def test_rope_special_values_stay_in_their_pair():
    x = torch.zeros((1, 1, 16), device="cuda")
    x[0, 0, 1], x[0, 0, 14], x[0, 0, 15] = math.inf, math.nan, -math.inf
    y = torch.empty_like(x)
    for layout, hit in (("half", [1, 5]), ("interleaved", [0, 1])):
        att.rope_apply(att.rope_encode(8, layout), tensor_map(x, "f32"), tensor_map(y, "f32"), ints([5]), False,
                       stream())
        bad = (~torch.isfinite(y[0, 0])).nonzero()[:, 0].tolist()
        assert bad == hit + [14, 15]


# ---- append ------------------------------------------------------------------------

def make_pool(shape, dtype, heads_first, g, gap=0):
    """[pages, slots, heads, dim] view of a pool in either order, with gaps."""
    pages, slots, n, dim = shape
    order = (pages, n, slots, dim) if heads_first else shape
    whole, v = padded(order, dtype, gap, g)
    return whole, (v.transpose(1, 2) if heads_first else v)


def pool_map(v, dtype):
    return tensor_map(v.transpose(1, 2), dtype)          # dims (dim, slots, heads, pages)


@pytest.mark.parametrize("case", range(7))
def test_append(case):
    dtype, tokens, heads, kv, dim, rot, layout, slots, first, gap = [
        ("bf16", 1, 4, 1, 64, 64, "half", 16, False, 0), ("f16", 9, 8, 2, 128, 128, "half", 7, True, 8),
        ("bf16", 1031, 6, 3, 96, 40, "interleaved", 48, False, 0), ("f32", 33, 2, 2, 80, 30, "half", 1, True, 0),
        ("f16", 12, 0, 2, 100, 100, "half", 256, False, 0), ("bf16", 10, 5, 5, 256, 0, "half", 16, False, 8),
        ("bf16", 700, 1, 4, 72, 72, "interleaved", 5, True, 0)][case]
    g = gen(100 + case)
    rows, row_pages = 5, -(-tokens // slots) + 2
    pages = rows * row_pages + 3
    kw, kp = make_pool((pages, slots, kv, dim), dtype, first, g, gap)
    vw, vp = make_pool((pages, slots, kv, dim), dtype, not first, g, gap)
    table = torch.randperm(pages, generator=g)[:rows * row_pages].view(rows, row_pages).to(torch.int32)
    wide = torch.full((rows, row_pages + 3), -7, dtype=torch.int32)
    wide[:, :row_pages] = table
    wide = wide.cuda()
    _, q = padded((tokens, max(heads, 1), dim), dtype, 0, g)
    _, k = padded((tokens, kv, dim), dtype, 8, g)
    _, v = padded((tokens, kv, dim), dtype, 0, g)
    q_out = torch.empty_like(q)
    spots = torch.randperm(rows * row_pages * slots, generator=g)[:tokens].numpy()
    row, at = spots // (row_pages * slots), spots % (row_pages * slots)
    if tokens > 4:
        row[3] = -1                                       # padding
    pos = torch.randint(0, 70000, (tokens,), generator=g).numpy()
    plan = att.rope_encode(rot, layout) if rot else None
    pt = att.page_table(wide[:, :row_pages], None, None, pages, slots)
    old_k, old_v = f64(kp), f64(vp)
    junk = [w.clone() for w in (kw, vw)]
    use_q = heads > 0
    att.rope_append(plan, tensor_map(q, dtype) if use_q else None, tensor_map(q_out, dtype) if use_q else None,
                    tensor_map(k, dtype), tensor_map(v, dtype), pool_map(kp, dtype), pool_map(vp, dtype), pt, ints(row),
                    ints(at), ints(pos) if rot else 0, stream())
    th = ok.rope_thetas(rot) if rot else []
    if use_q:
        want, size = ok.rope(f64(q), pos, th, layout)
        assert (np.abs(f64(q_out) - want) <= rope_limit(want, size, dtype)).all()
    want, size = ok.rope(f64(k), pos, th, layout)
    lim = rope_limit(want, size, dtype)
    lim_pool = np.zeros(old_k.shape)
    for t in range(tokens):
        if row[t] < 0:
            continue
        page, slot = int(table[row[t], at[t] // slots]), at[t] % slots
        old_k[page, slot], old_v[page, slot] = want[t], f64(v)[t]
        lim_pool[page, slot] = lim[t] if rot else 0
    assert (np.abs(f64(kp) - old_k) <= lim_pool).all()
    assert np.array_equal(f64(vp), old_v)
    if gap:
        for w, o in zip((kw, vw), junk):
            assert torch.equal(w[..., dim:].contiguous().view(torch.uint8).cpu(),
                               o[..., dim:].contiguous().view(torch.uint8).cpu())


def test_append_skips_what_is_out_of_range():
    g = gen(5)
    _, kp = make_pool((4, 4, 1, 64), "bf16", False, g)
    k = torch.randn((6, 1, 64), generator=g).to(torch.bfloat16).cuda()
    table = ints([[0, 9], [-1, 2]])
    pt = att.page_table(table, None, None, 4, 4)
    old = kp.clone()
    # page 9 of 4, entry -1, row 2 of 2, token index past the row, a negative index; the last token is right
    att.rope_append(None, None, None, tensor_map(k, "bf16"), tensor_map(k, "bf16"), pool_map(kp, "bf16"),
                    pool_map(kp, "bf16"), pt, ints([0, 1, 2, 0, 0, 1]), ints([4, 0, 0, 8, -1, 7]), 0, stream())
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    old[2, 3] = k[5]
    assert torch.equal(kp, old)


# ---- pages ---------------------------------------------------------------------------

def same(pt_t, lens, refs, pools, want):
    assert np.array_equal(pt_t.cpu().numpy(), want.table)
    assert np.array_equal(lens.cpu().numpy(), want.lens)
    assert np.array_equal(refs.cpu().numpy(), want.refs)
    for p, w in zip(pools, want.pools):
        assert np.array_equal(p.cpu().numpy(), w)


@pytest.mark.parametrize("case", range(8))
def test_pages_random_steps(case):
    """Random extends, forks, frees and compactions, against the oracle after
    each: exact, shortages included."""
    slots, pages, rows, row_pages, npool, dim, dtype, first = [
        (4, 40, 6, 5, 1, 16, "u16", False), (1, 100, 20, 9, 2, 8, "u16", True), (16, 70, 8, 300, 3, 24, "u16", False),
        (7, 3000, 40, 70, 2, 8, "u8", True), (3, 67000, 12, 3000, 1, 8, "u16", False), (5, 1, 3, 2, 2, 8, "u16", False),
        (2, 65536, 9, 1100, 1, 8, "u16", True), (48, 200, 10, 20, 1, 40, "u8", False)][case]
    rng = np.random.default_rng(case)
    heads = 2
    shape = (pages, heads, slots, dim) if first else (pages, slots, heads, dim)
    g = gen(case)
    if dtype == "u8":
        dim *= 2
        shape = shape[:-1] + (dim,)
        pools = [torch.randint(0, 256, shape, generator=g).to(torch.uint8).cuda() for _ in range(npool)]
    else:
        pools = [torch.randint(-999, 999, shape, generator=g).to(torch.int16).cuda() for _ in range(npool)]
    maps = att.tmap_array([tensor_map(p if first else p.transpose(1, 2), dtype) for p in pools])
    wide = torch.full((rows, row_pages + 1), -5, dtype=torch.int32, device="cuda")
    table, lens, refs = wide[:, :row_pages], ints([0] * rows), ints([0] * pages)
    table.fill_(-1)
    want = ok.Pages(table.cpu().numpy(), lens.cpu().numpy(), refs.cpu().numpy(), slots,
                    [p.cpu().numpy() for p in pools])
    pt = att.page_table(table, lens, refs, pages, slots)
    ws = torch.empty(att.page_workspace(pt, rows), dtype=torch.uint8, device="cuda")
    room = slots * row_pages
    for step in range(24):
        what = rng.choice(["extend", "extend", "fork", "free", "compact"]) if step else "extend"
        empty = [r for r in range(rows) if want.lens[r] == 0]
        held = [r for r in range(rows) if want.lens[r] > 0]
        if what == "extend":
            n = int(rng.integers(1, rows + 1))
            who = rng.permutation(rows)[:n]
            add = rng.integers(0, max(2, min(room, 3 * pages * slots // rows)), n)
            flag = ints([9] * n)
            att.page_extend(pt, ints(who), ints(add), n, flag, ws, stream())
            assert flag.cpu().tolist() == want.extend(who.tolist(), add.tolist())
        elif what == "fork" and empty and held:
            n = int(rng.integers(1, len(empty) + 1))
            src, dst = rng.choice(held, n), rng.permutation(empty)[:n]
            flag = ints([9] * n)
            att.page_fork(pt, maps, ints(src), ints(dst), n, flag, ws, stream())
            assert flag.cpu().tolist() == want.fork(src.tolist(), dst.tolist())
        elif what == "free":
            who = rng.choice(rows, int(rng.integers(1, rows + 1)))       # some twice
            att.page_free(pt, ints(who), len(who), stream())
            want.free(who.tolist())
        elif what == "compact":
            used = ints([-1])
            if step % 2:
                att.page_compact(pt, pt, maps, used, ws, stream())
            else:
                t2, r2 = torch.full_like(table, -3), torch.full_like(refs, -3)
                old_t, old_r = table.clone(), refs.clone()
                att.page_compact(pt, att.page_table(t2, lens, r2, pages, slots), maps, used, ws, stream())
                assert torch.equal(table, old_t) and torch.equal(refs, old_r)
                table.copy_(t2)
                refs.copy_(r2)
            assert used.item() == want.compact()
        same(table, lens, refs, pools, want)
        assert (wide[:, row_pages:] == -5).all()


def test_page_copy_strided_pools():
    """Pages with gaps between heads, tokens and pages, rows that are not whole
    16 bytes, skipped entries, a part boundary inside a page."""
    g = gen(9)
    for slots, heads, dim, dtype, gap in [(5, 3, 20, "u8", 12), (100, 5, 33, "u16", 7), (256, 4, 128, "u16", 0),
                                          (3, 1, 16, "u8", 0)]:
        n = 16 // (1 if dtype == "u8" else 2)
        wide = -(-(dim + gap) // n) * n
        t = torch.randint(0, 200, (9, slots, heads, wide), generator=g).to(TORCH[dtype]).cuda()
        other = torch.randint(0, 200, (9, slots, heads, wide), generator=g).to(TORCH[dtype]).cuda()
        src, dst = [0, -1, 4, 7, 2], [1, 3, 5, -1, 8]
        wants = []
        for x in (t, other):
            w = x.clone()
            for a, b in zip(src, dst):
                if a >= 0 and b >= 0:
                    w[b, ..., :dim] = w[a, ..., :dim]
            wants.append(w)
        maps = [pool_map(x[..., :dim], dtype) for x in (t, other)]
        att.page_copy(maps, ints(src), ints(dst), 5, stream())
        assert torch.equal(t, wants[0]) and torch.equal(other, wants[1])


def test_pages_refuse_in_the_kernel():
    """Rows and pages out of range, negative lengths and growth, destinations
    in use: not served, nothing else touched, the error recorded."""
    table, lens, refs = ints([[0, 1], [-1, -1], [7, -1]]), ints([5, 0, 2]), ints([1, 1, 0, 0])
    pt = att.page_table(table, lens, refs, 4, 4)
    ws = torch.empty(att.page_workspace(pt, 8), dtype=torch.uint8, device="cuda")
    keep = [x.clone() for x in (table, lens, refs)]

    def recorded():
        with pytest.raises(att.TmapError) as e:
            att.tile_device_status(stream())
        assert e.value.name == "ERR_PAGE"

    flag = ints([9] * 4)
    att.page_extend(pt, ints([3, -1, 0, 0]), ints([1, 1, -1, 100]), 4, flag, ws, stream())
    recorded()
    assert flag.cpu().tolist() == [0, 0, 0, 0]
    att.page_fork(pt, None, ints([0, 5, 0, 0]), ints([2, 1, -2, 3]), 4, flag, ws, stream())
    recorded()
    assert flag.cpu().tolist() == [0, 0, 0, 0]
    att.page_free(pt, ints([3]), 1, stream())
    recorded()
    for x, w in zip((table, lens, refs), keep):
        assert torch.equal(x, w)
    att.page_free(pt, ints([2]), 1, stream())              # page 7 of 4: dropped from the row
    recorded()
    assert table.cpu().tolist() == [[0, 1], [-1, -1], [-1, -1]] and torch.equal(refs, keep[2])
    pools = torch.zeros((4, 4, 1, 8), dtype=torch.int16, device="cuda")
    att.page_copy(pool_map(pools, "u16"), ints([0, 4]), ints([9, 1]), 2, stream())
    recorded()


# ---- attention -------------------------------------------------------------------------

ATTN = [  # dtype, batch, q_len, heads, kv, dim, slots, prefix, lens, heads_first, gap
    ("bf16", 1, 1, 1, 1, 64, 16, 0, [1], False, 0),
    ("bf16", 2, 1, 4, 2, 128, 16, 37, [0, 70], False, 0),
    ("f16", 3, 1, 8, 2, 64, 7, 130, [5, 0, 33], True, 8),
    ("f16", 3, 3, 6, 3, 80, 16, 65, [2, 3, 40], False, 0),
    ("bf16", 4, 5, 10, 2, 96, 48, 200, [5, 4, 0, 257], True, 0),
    ("bf16", 5, 2, 5, 1, 256, 1, 31, [64, 32, 1, 2, 100], False, 0),
    ("f16", 2, 1, 16, 1, 128, 256, 1000, [500, 300], False, 0),
    ("bf16", 2, 4, 2, 2, 192, 5, 0, [0, 3], False, 0),
    ("bf16", 33, 1, 8, 2, 64, 32, 129, [(7 * i) % 50 for i in range(33)], True, 0),
    ("f16", 70, 2, 2, 1, 128, 16, 257, [(11 * i) % 90 for i in range(70)], False, 0),
    ("bf16", 9, 17, 4, 4, 40, 3, 66, [20 + i for i in range(9)], False, 0),
    ("f16", 1, 1, 64, 1, 8, 9, 100, [3], False, 0),
    ("bf16", 130, 1, 2, 2, 128, 64, 512, [i % 3 for i in range(130)], True, 0),
    ("bf16", 3, 40, 3, 1, 128, 16, 100, [300, 40, 41], False, 0),
]


def attn_setup(case, g, spare=2):
    dtype, batch, q_len, heads, kv, dim, slots, prefix, lens, first, gap = case
    shared = -(-prefix // slots)
    each = [-(-n // slots) for n in lens]
    pages = shared + sum(each) + spare
    _, kp = make_pool((pages, slots, kv, dim), dtype, first, g, gap)
    _, vp = make_pool((pages, slots, kv, dim), dtype, first, g, gap)
    order = torch.randperm(pages, generator=g).tolist()
    row_pages = max([shared, 1] + each)
    table = np.full((batch + 2, row_pages), -1, dtype=np.int32)
    table[1, :shared] = order[:shared]
    rows = [(b + 3) % (batch + 1) for b in range(batch)]
    rows = [r if r < 1 else r + 1 for r in rows]
    rows = list(dict.fromkeys(rows))
    assert len(rows) == batch and 1 not in rows
    at = shared
    full = np.zeros(batch + 2, dtype=np.int32)
    full[1] = prefix
    for b in range(batch):
        table[rows[b], :each[b]] = order[at:at + each[b]]
        full[rows[b]] = lens[b]
        at += each[b]
    _, q = padded((batch, q_len, heads, dim), dtype, gap, g)
    return q, kp, vp, table, full, rows


def attn_run(q, kp, vp, table, lens, rows, slots, prefix, scale, dtype, hint=100, lse=True):
    o = torch.full_like(q, float("nan"))
    l = torch.full(q.shape[:3], float("nan"), device="cuda")
    mq, mk = tensor_map(q, dtype), pool_map(kp, dtype)
    pt = att.page_table(ints(table), ints(lens), None, kp.shape[0], slots)
    ws = torch.full((att.attn_workspace(mq, mk, prefix, hint),), 255, dtype=torch.uint8, device="cuda")
    d_table, d_lens = ints(table), ints(lens)
    pt = att.page_table(d_table, d_lens, None, kp.shape[0], slots)
    d_rows = ints(rows) if rows is not None else 0
    att.attn_shared_prefix(mq, mk, pool_map(vp, dtype), pt, 1, prefix, d_rows, hint, scale, tensor_map(o, dtype),
                           l if lse else 0, ws, stream())
    torch.cuda.synchronize()
    return f64(o), f64(l)


def attn_check(got, got_lse, q, kp, vp, table, lens, rows, slots, prefix, scale, dtype):
    dim = q.shape[-1]
    want, lse, weight, size, n = ok.attention(f64(q), f64(kp), f64(vp), table, lens, slots, 1, prefix, rows, scale)
    shift = (dim + 8) * 2.0 ** -24 * size + 2.0 ** -21
    n = n[..., None]
    limit = weight * (ok.half_step(dtype) + 2 * shift[..., None] + (n + 32) * 2.0 ** -24)
    limit += ok.half_step(dtype) * np.abs(want) + (n + 1) * (2.0 ** -25 if dtype == "f16" else 1e-37) * 8
    assert (np.abs(got - want) <= limit).all(), (np.abs(got - want) - limit).max()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and (got[empty] == 0).all()
    with np.errstate(invalid="ignore"):
        off = np.abs(got_lse - lse)[~empty]
    assert (off <= (shift + (n[..., 0] + 32) * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse))[~empty]).all()


@pytest.mark.parametrize("hint", [0, 100, 5000])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case, hint):
    c = ATTN[case]
    dtype, slots, prefix = c[0], c[6], c[7]
    q, kp, vp, table, lens, rows = attn_setup(c, gen(200 + case))
    scale = 1.0 / math.sqrt(c[5])
    got, lse = attn_run(q, kp, vp, table, lens, rows, slots, prefix, scale, dtype, hint)
    attn_check(got, lse, q, kp, vp, table, lens, rows, slots, prefix, scale, dtype)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 6.0])
def test_attention_scales(scale):
    c = ("f16", 3, 1, 4, 2, 64, 16, 90, [40, 0, 17], False, 0)
    q, kp, vp, table, lens, rows = attn_setup(c, gen(31))
    got, lse = attn_run(q, kp, vp, table, lens, rows, 16, 90, scale, "f16")
    attn_check(got, lse, q, kp, vp, table, lens, rows, 16, 90, scale, "f16")


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("prefix", [0, 45, 300])
def test_attention_ignores_what_it_does_not_see(prefix, q_len):
    """NaN and infinities in every slot past the lengths, in pages of others,
    and in tokens that come after a query, reach no query that does not see
    them."""
    c = ("bf16", 5, q_len, 8, 2, 128, 16, prefix, [9, 0, 40, 33, 64], False, 0)
    g = gen(77)
    q, kp, vp, table, lens, rows = attn_setup(c, g)
    clean = attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.1, "bf16")
    attn_check(*clean, q, kp, vp, table, lens, rows, 16, prefix, 0.1, "bf16")
    seen = torch.zeros(kp.shape[:2], dtype=torch.bool)
    for r in [1] + rows:
        for t in range(int(lens[r])):
            seen[table[r][t // 16], t % 16] = True
    for pool in (kp, vp):
        pool[(~seen).cuda()] = float("nan")
    vp[0][(~seen)[0].cuda()] = float("inf")
    got = attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.1, "bf16")
    assert np.array_equal(got[0], clean[0]) and np.array_equal(got[1], clean[1])
    if q_len > 1:                                          # the last token of a row is seen by its last query alone
        for value in (float("nan"), float("inf")):
            for r in rows:
                if lens[r]:
                    t = int(lens[r]) - 1
                    kp[table[r][t // 16], t % 16] = value
                    vp[table[r][t // 16], t % 16] = value
            got = attn_run(q, kp, vp, table, lens, rows, 16, prefix, 0.1, "bf16")
            assert np.array_equal(got[0][:, :-1], clean[0][:, :-1])
            assert np.array_equal(got[1][:, :-1], clean[1][:, :-1])


def test_attention_without_rows_or_lse_and_shared_pages():
    """d_rows NULL is rows 0, 1, ...; two sequences may hold the same pages;
    lse is optional."""
    g = gen(8)
    _, kp = make_pool((6, 16, 1, 64), "f16", False, g)
    _, vp = make_pool((6, 16, 1, 64), "f16", False, g)
    table, lens = np.array([[3, 1], [5, 0], [3, 4]], dtype=np.int32), np.array([30, 20, 18], dtype=np.int32)
    q = torch.randn((3, 1, 2, 64), generator=g).to(torch.float16).cuda()
    got, lse = attn_run(q, kp, vp, table, lens, None, 16, 20, 0.125, "f16")
    attn_check(got, lse, q, kp, vp, table, lens, None, 16, 20, 0.125, "f16")
    again, none = attn_run(q, kp, vp, table, lens, None, 16, 20, 0.125, "f16", lse=False)
    assert np.array_equal(got, again) and np.isnan(none).all()


def test_attention_skips_bad_pages():
    """Entries that are not pages, lengths past the row and rows out of range:
    their keys count as not there, the error is recorded."""
    g = gen(12)
    _, kp = make_pool((4, 16, 1, 64), "bf16", False, g)
    _, vp = make_pool((4, 16, 1, 64), "bf16", False, g)
    q = torch.randn((3, 1, 1, 64), generator=g).to(torch.bfloat16).cuda()
    table, lens = np.array([[0, 4], [3, -1], [1, 2]], dtype=np.int32), np.array([32, 20, 99], dtype=np.int32)
    got, lse = attn_run(q, kp, vp, table, lens, [0, 2, 7], 16, 20, 0.125, "bf16")
    with pytest.raises(att.TmapError) as e:
        att.tile_device_status(stream())
    assert e.value.name == "ERR_PAGE"
    # the keys that are left: the prefix's first page; 16 tokens of row 0; the 32 that row 2 has room for
    attn_check(got, lse, q, kp, vp, np.array([[0, -1], [3, -1], [1, 2], [0, 0]]), np.array([16, 16, 32, 0]), [0, 2, 3],
               16, 16, 0.125, "bf16")


# ---- streams, graphs, large offsets ---------------------------------------------------------

def test_other_stream_and_graph_replays():
    """A decode step captured once and replayed while lengths, tables and
    inputs change in place, with eager work between the replays: every replay
    equals the eager call on the same state."""
    g = gen(21)
    c = ("bf16", 4, 1, 8, 2, 128, 16, 150, [20, 0, 33, 64], False, 0)
    batch, heads, kv, dim, slots, prefix = 4, 8, 2, 128, 16, 150
    q, kp, vp, table, lens, rows = attn_setup(c, g, spare=40)
    row_pages = 12
    wide = np.full((len(table), row_pages), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table[:, :row_pages]
    t, l = ints(wide), ints(lens)
    refs = torch.zeros(kp.shape[0], dtype=torch.int32)
    for p in wide[wide >= 0]:
        refs[p] += 1
    refs = refs.cuda()
    pt = att.page_table(t, l, refs, kp.shape[0], slots)
    d_rows, one = ints(rows), ints([1] * batch)
    flag = ints([0] * batch)
    x = torch.zeros((batch, heads, dim), dtype=torch.bfloat16, device="cuda")
    xk, xv = (torch.zeros((batch, kv, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    turned, o = torch.empty_like(x), torch.empty_like(x)
    lse = torch.empty((batch, heads), device="cuda")
    at, pos = ints([0] * batch), ints([0] * batch)
    plan = att.rope_encode(dim)
    q4 = turned.view(batch, 1, heads, dim)
    mq, mk, mv = tensor_map(q4, "bf16"), pool_map(kp, "bf16"), pool_map(vp, "bf16")
    ws = torch.empty(att.page_workspace(pt, batch), dtype=torch.uint8, device="cuda")
    aws = torch.empty(att.attn_workspace(mq, mk, prefix, 64), dtype=torch.uint8, device="cuda")
    maps = [tensor_map(i, "bf16") for i in (x, turned, xk, xv)]
    mo = tensor_map(o.view(batch, 1, heads, dim), "bf16")

    def step(st):
        at.copy_(l[d_rows.long()])
        torch.add(at, prefix, out=pos)
        att.page_extend(pt, d_rows, one, batch, flag, ws, st)
        att.rope_append(plan, *maps, mk, mv, pt, d_rows, at, pos, st)
        att.attn_shared_prefix(mq, mk, mv, pt, 1, prefix, d_rows, 64, dim ** -0.5, mo, lse, aws, st)

    state = [t, l, refs, kp, vp]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [s.clone() for s in state]
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(torch.cuda.current_stream().cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for s, k in zip(state, saved):
        s.copy_(k)
    for i in range(5):
        for inp in (x, xk, xv):
            inp.copy_(torch.randn(inp.shape, generator=g).to(torch.bfloat16))
        now = [s.clone() for s in state]
        step(stream())
        torch.cuda.synchronize()
        eager = [s.clone() for s in state + [turned, o, lse, flag]]
        for s, k in zip(state, now):
            s.copy_(k)
        for out in (turned, o, lse, flag):
            out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, state + [turned, o, lse, flag]):
            assert torch.equal(a, b), i
        assert flag.cpu().tolist() == [1] * batch


def test_offsets_past_32_bits():
    """Pages at byte offsets past 4 GiB: appended, copied, compacted and
    attended to."""
    slots, kv, dim, pages = 256, 8, 128, 10000                  # 512 KiB a page, 4.9 GiB a pool
    kp = torch.empty((pages, slots, kv, dim), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty((pages, slots, kv, dim), dtype=torch.bfloat16, device="cuda")
    g = gen(4)
    far = [9998, 9000, 8500]
    assert far[2] * slots * kv * dim * 2 > 2 ** 32
    for p in far:
        kp[p].copy_(torch.randn((slots, kv, dim), generator=g).to(torch.bfloat16))
        vp[p].copy_(torch.randn((slots, kv, dim), generator=g).to(torch.bfloat16))
    maps = att.tmap_array([pool_map(kp, "bf16"), pool_map(vp, "bf16")])
    att.page_copy(maps, ints([9998]), ints([9999]), 1, stream())
    assert torch.equal(kp[9999], kp[9998]) and torch.equal(vp[9999], vp[9998])
    k = torch.randn((1, kv, dim), generator=g).to(torch.bfloat16).cuda()
    table, lens = ints([[9000, 8500], [9999, -1]]), ints([300, 41])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    for p in (9000, 8500, 9999):
        refs[p] = 1
    pt = att.page_table(table, lens, refs, pages, slots)
    att.rope_append(None, None, None, tensor_map(k, "bf16"), tensor_map(k, "bf16"), maps[0], maps[1], pt, ints([1]),
                    ints([40]), 0, stream())
    assert torch.equal(kp[9999, 40], k[0]) and torch.equal(vp[9999, 40], k[0])
    q = torch.randn((1, 1, 16, dim), generator=g).to(torch.bfloat16).cuda()
    mq = tensor_map(q, "bf16")
    o, lse = torch.empty_like(q), torch.empty((1, 1, 16), device="cuda")
    aws = torch.empty(att.attn_workspace(mq, maps[0], 300, 41), dtype=torch.uint8, device="cuda")
    ws = torch.empty(att.page_workspace(pt, 0), dtype=torch.uint8, device="cuda")
    small_k, small_v = (torch.stack([p[9000], p[8500], p[9999]]) for p in (kp, vp))
    for _ in range(2):                                          # before and after the pages move to 0, 1, 2
        att.attn_shared_prefix(mq, maps[0], maps[1], pt, 0, 300, ints([1]), 41, 0.1, tensor_map(o, "bf16"), lse, aws,
                               stream())
        want, _, weight, *_ = ok.attention(f64(q), f64(small_k), f64(small_v), np.array([[0, 1], [2, -1]]),
                                           np.array([300, 41]), slots, 0, 300, [1], 0.1)
        assert (np.abs(f64(o) - want) <= 2.0 ** -8 * (weight + np.abs(want)) + 1e-4 * weight).all()
        att.page_compact(pt, pt, maps, 0, ws, stream())
        assert sorted(table.flatten().tolist()) == [-1, 0, 1, 2]
