"""Attention over the cache where most of the weights are far below the largest one.

A weight is rounded to the element type.  Beside that of its last bit, an f16 weight
below 2^-14 of what weights are taken relative to, times 2^7, has an error of half a
step of the smallest numbers: 2^-25 * 2^-7 of the largest weight.  n of them shift a
result by n * 2^-32 of the largest value at most."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native  # noqa: E402
from test_gpu_attn_cache import FAR, Setup, parents_of  # noqa: E402
from test_gpu_kvcache import f64, gen, ints  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


def check(s, window=0, sinks=0, parents=None, scale=1.0, hint=None):
    got, got_lse = s.run(window, sinks, None if parents is None else ints(parents), scale, hint=hint)
    q, step = f64(s.q), ok.half_step(s.dtype)
    for b, length in enumerate(s.seq_lens):
        k, v = s.tokens(s.k, b), s.tokens(s.v, b)
        sees = ok.causal_sees(length, s.q_len, window, sinks) if parents is None else \
            ok.tree_sees(length, [int(p) for p in parents[b]], window, sinks)
        want, lse, weight, size, n = ok.attend(q[b], k, v, sees, scale)
        shift = ((s.dim + 8) * 2.0 ** -24 * size + 2.0 ** -21)[..., None]
        limit = weight * (step + 2 * shift + (n[..., None] + 32) * 2.0 ** -24) + step * np.abs(want)
        if s.dtype == "f16":
            limit += n[..., None] * 2.0 ** -32 * np.abs(v).max()
        off = np.abs(got[b] - want)
        assert (off <= limit).all(), (b, (off / limit).max())
        near = shift[..., 0] + (n + 32) * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse)
        assert (np.abs(got_lse[b] - lse) <= near).all()
    return want


def one_far_above(s, by):
    """Every sequence's first token scores `by` for each query (at scale 1), all the others nearly 0; its values are 0
    and theirs are not negative, so that they make the result together."""
    s.q.zero_()
    s.q[..., 0] = 4.0
    for p in (s.k, s.v):
        x = p if s.heads_first else p.transpose(1, 2)                    # [pages, kv, rows, dim]
        if s.fmt == "same":
            if p is s.k:
                x[..., 0] *= 0.03
            else:
                x.abs_()
            continue
        tail = torch.zeros((*x.shape[:2], (x.shape[2] - s.slots) * s.dim), dtype=torch.uint8)
        tail[..., :2 * s.slots] = torch.full((*x.shape[:2], s.slots), 1 / 64).bfloat16().view(torch.uint8)
        x[:, :, s.slots:] = tail.view(*x.shape[:2], -1, s.dim).cuda()
        if p is s.k:
            x[:, :, :s.slots, 0] &= 1 if s.fmt == "int8" else 0x2F
        else:
            x[:, :, :s.slots] &= 0x7F
    for r in s.rows:
        page = int(s.table[r, 0])
        for p in (s.k, s.v):
            x = p[page] if s.heads_first else p[page].transpose(0, 1)    # [kv, rows, dim]
            if s.fmt == "same":
                x[:, 0] = 0
                if p is s.k:
                    x[:, 0, 0] = by / 4
                continue
            x[:, 0] = 0
            if p is s.k:                                                 # the code 64 times by / 256
                x[:, 0, 0] = 64 if s.fmt == "int8" else 0x68
            x[:, s.slots, :2] = torch.tensor([by / 256]).bfloat16().view(torch.uint8).cuda()


@pytest.mark.parametrize("by", [9.0, 17.5, 20.0])
@pytest.mark.parametrize("fmt", ["same", "int8", "e4m3"])
@pytest.mark.parametrize("q_len,hint", [(1, None), (3, 100), (70, FAR), (150, 100)])
def test_many_small_weights(q_len, hint, fmt, by):
    s = Setup(gen(800), "f16", fmt, [40000], None, q_len, 2, 1, 64, 64)
    one_far_above(s, by)
    want = check(s, hint=hint)
    assert np.abs(want).min() > 0.1 * 39850 * math.exp(-by) / (1 + 40000 * math.exp(-by))   # the small ones make it


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_len,hint", [(1, None), (1, 100), (80, FAR), (80, 100)])
def test_a_sink_far_above_all(q_len, hint, dtype):
    """131072 tokens 17.5 below one whose value is 0 are 0.3 % of a result of ones."""
    s = Setup(gen(801), dtype, "same", [131073], None, q_len, 1, 1, 64, 128)
    s.k.zero_(), s.v.fill_(1.0)
    one_far_above(s, 17.5)
    want = check(s, hint=hint)
    n = 131073 - q_len
    assert abs(want[0, 0, 0] - n * math.exp(-17.5) / (1 + n * math.exp(-17.5))) < 1e-9


@pytest.mark.parametrize("dim,fmt", [(64, "same"), (96, "same"), (128, "int8"), (128, "e4m3"), (192, "same"), (256, "int8")])
@pytest.mark.parametrize("q_len,hint", [(2, None), (100, 100), (100, FAR)])
def test_scores_of_all_sizes(q_len, hint, dim, fmt):
    """Scores whose spread leaves most weights below f16's normal numbers; windows, sinks and a tree."""
    g = gen(802)
    s = Setup(g, "f16", fmt, [900, 300], None, q_len, 4, 2, dim, 16)
    check(s, 0, 0, None, 5 / math.sqrt(dim), hint)
    check(s, 120, 3, None, -3 / math.sqrt(dim), hint)
    check(s, 0, 0, parents_of(g, 2, q_len, "near"), 5 / math.sqrt(dim), hint)


def scales_of(p, s, scale):
    """All scales of a pool of codes."""
    x = p if s.heads_first else p.transpose(1, 2)
    tail = torch.zeros((*x.shape[:2], (x.shape[2] - s.slots) * s.dim), dtype=torch.uint8)
    tail[..., :2 * s.slots] = torch.full((*x.shape[:2], s.slots), scale).bfloat16().view(torch.uint8)
    x[:, :, s.slots:] = tail.view(*x.shape[:2], -1, s.dim).cuda()


@pytest.mark.parametrize("fmt", ["same", "int8", "e4m3"])
@pytest.mark.parametrize("q_len,heads,tile", [(1, 1, 128), (40, 1, 128), (200, 16, 64)])
@pytest.mark.parametrize("power", [12, 14, 16, 17, 18, 20, 23])
def test_scores_so_large_that_their_roundings_count(power, q_len, heads, tile, fmt):
    """Scores of 2^power that pass the largest of before by about 2^8, tile after tile (every fourth of 32, or each of 64):
    every weight is a number that f16 holds, beside the largest rest of a value's scale too, and a result lies among the
    values."""
    n, units = 1500, 2.0 ** np.arange(15, -9, -4)
    s = Setup(gen(803), "f16", fmt, [n] * 6, None, q_len, heads, 1, 64, 16)
    scale = max(1.0, 2.0 ** (power - 17))
    x = torch.rand((6, n), generator=gen(804)).numpy()
    want = (2.0 ** power + 8 * (np.arange(n) // tile) + 0.1 * (x - 0.5)) * math.log(2) / scale
    s.q.zero_()
    s.q[..., :6] = torch.from_numpy(units).half().cuda()
    for b, r in enumerate(s.rows):
        rest, digits = want[b], np.zeros((n, 6))
        for d, unit in enumerate(units):                                 # 0 .. 15, which every format holds
            digits[:, d] = np.floor(rest / unit)
            rest = rest - digits[:, d] * unit
        assert digits.min() >= 0 and digits.max() < 16
        page, slot = s.table[r].cpu().numpy()[np.arange(n) // 16], np.arange(n) % 16
        code = torch.from_numpy(digits)
        code = code.half() if fmt == "same" else code.to(torch.int8).view(torch.uint8) if fmt == "int8" else \
            code.float().to(torch.float8_e4m3fn).view(torch.uint8)
        s.k[page, slot] = 0
        s.k[page, slot, 0, :6] = code.cuda()
    if fmt != "same":
        scales_of(s.k, s, 1.0), scales_of(s.v, s, 1.9921875 / 64)
    got, lse = s.run(0, 0, None, scale, hint=100)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    for b in range(6):
        assert (np.abs(got[b]) <= np.abs(s.tokens(s.v, b)).max() * (1 + 2.0 ** -9)).all()
