"""The cache's calls together on pools of codes, against what the cache holds.

Each step's new tokens are read from the pools as soon as they are written, and
compared with the keys and values that were written: within half a code.  From
then on the test's record holds the codes' numbers, so that attention is held to
the limits of its own roundings (test_gpu_attn_cache): the wrong token, head or
window is far outside of them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native, stream  # noqa: E402
from test_gpu_attn_cache import parents_of  # noqa: E402
from test_gpu_cache_steps import Cache  # noqa: E402
from test_gpu_kvcache import TORCH, f64, gen, ints, tensor_map  # noqa: E402


def limits(dtype, q, k, v, sees, scale):
    """What attention over these tokens is, and how far a result and its lse may be off.  An f16 weight has an error of
    2^-32 beside that of its last bit."""
    step = ok.half_step(dtype)
    want, lse, weight, size, n = ok.attend(q, k, v, sees, scale)
    shift = (q.shape[-1] + 8) * 2.0 ** -24 * size + 2.0 ** -21
    n = n[..., None]
    limit = weight * (step + 2 * shift[..., None] + (n + 32) * 2.0 ** -24) + step * np.abs(want)
    limit += (n + 1) * (2.0 ** -32 if dtype == "f16" else 0.0) * np.abs(v).max(initial=0.0)
    return want, limit, lse, shift + (n[..., 0] + 32) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


class Codes(Cache):
    def held(self, i, r, at):
        """Tokens `at` of row r as pool i holds them: codes and scales, [n, kv, dim] and [n, kv]."""
        page = self.table[r].cpu().numpy()[at // self.slots]
        code, scale = ok.split_codes(self.pools[i][torch.from_numpy(page).long().cuda()].cpu().numpy()
                                     .transpose(0, 2, 1, 3), self.slots, self.fmt)
        n = np.arange(len(at))
        return code[n, :, at % self.slots], scale[n, :, at % self.slots]

    def append(self, rows, pos, q, k, v):
        start = {r: len(self.record[r]) for r in rows}
        out = super().append(rows, pos, q, k, v)
        n = q.shape[1]
        for i, r in enumerate(rows):
            at = np.arange(start[r], start[r] + n)
            new = []
            for which, (x, turned) in enumerate(((k, True), (v, False))):
                y, size = f64(x)[i], np.abs(f64(x)[i])
                if turned:
                    y, size = ok.rope(f64(x)[i], pos[i], self.thetas)
                code, s = self.held(which, r, at)
                off = size * 2.0 ** -21 if turned else 0 * size
                top = np.abs(y).max(-1) / ok.LARGEST[self.fmt]
                assert (s >= top - off.max(-1)).all()
                assert (s <= (top + off.max(-1)) * (1 + 2.0 ** -7) * (1 + 2.0 ** -23)).all()
                step = s[..., None] * ok.code_step(y / s[..., None] * (1 + 2.0 ** -20), self.fmt)
                got = code * s[..., None]
                assert (np.abs(got - y) <= step / 2 + off + 2.0 ** -24 * np.abs(y)).all()
                new.append(got)
            self.record[r][start[r]:] = list(zip(*new))
        return out

    def check(self, rows, q, o, lse, parents):
        for i, r in enumerate(rows):
            k, v = (np.stack([t[x] for t in self.record[r]]) for x in (0, 1))
            sees = ok.causal_sees(len(k), q.shape[1], self.window, self.sinks) if parents is None else \
                ok.tree_sees(len(k), [int(p) for p in parents[i]], self.window, self.sinks)
            want, limit, want_lse, near = limits(self.dtype, f64(q)[i], k, v, sees, 1 / math.sqrt(self.dim))
            off = np.abs(f64(o)[i] - want)
            assert (off <= limit).all(), (r, (off / limit).max())
            assert (np.abs(f64(lse)[i] - want_lse) <= near).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,window,sinks", [("int8", 40, 3), ("e4m3", 25, 2), ("int8", 0, 0), ("e4m3", 0, 0)])
@pytest.mark.parametrize("heads,kv,dim,slots", [(4, 2, 64, 8), (16, 2, 128, 16)])
def test_serving_codes(heads, kv, dim, slots, fmt, window, sinks, dtype):
    require_native()
    g, rng = gen(910), np.random.default_rng(4)
    c = Codes(dtype, fmt, 6, 200, slots, heads, kv, dim, window, sinks, g)

    def tokens(b, n):
        return [torch.randn((b, n, h, dim), generator=g).to(TORCH[dtype]).cuda() for h in (heads, kv, kv)]

    def causal(rows, n, hint=None):
        start = np.array([len(c.record[r]) for r in rows])
        c.attend(rows, c.append(rows, start[:, None] + np.arange(n), *tokens(len(rows), n)), hint=hint)

    def drafted(rows, n, most):
        parents = parents_of(g, len(rows), n, "near")
        depth = np.zeros((len(rows), n), int)
        for i in range(len(rows)):
            for j in range(n):
                depth[i, j] = 0 if parents[i, j] < 0 else depth[i, parents[i, j]] + 1
        base = np.array([len(c.record[r]) for r in rows])
        c.attend(rows, c.append(rows, base[:, None] + depth, *tokens(len(rows), n)), parents)
        keep, count = np.full((len(rows), most), -1), np.zeros(len(rows), int)
        for i in range(len(rows)):                                       # a way down the tree is accepted
            way = [int(rng.integers(0, n))]
            while parents[i, way[-1]] >= 0:
                way.append(int(parents[i, way[-1]]))
            way = way[::-1][:most]
            keep[i, :len(way)], count[i] = way, len(way)
        good = ints([0] * len(rows))
        att.page_keep(c.pt, c.all_maps, ints(rows), ints(base), ints(keep), ints(count), len(rows), good, stream())
        assert good.tolist() == [1] * len(rows)
        for i, r in enumerate(rows):
            c.record[r] = c.record[r][:base[i]] + [c.record[r][base[i] + k] for k in keep[i, :count[i]]]
        assert c.lens.tolist() == [len(t) for t in c.record]

    causal([0, 2, 4], 60)
    causal([0, 2, 4], 11, hint=1 << 20)
    for _ in range(2):
        causal([0, 2, 4], 1)
        drafted([4, 0, 2], 13, 5)
    good = ints([0, 0])
    att.page_fork(c.pt, c.all_maps, ints([2, 0]), ints([1, 5]), 2, good, c.ws, stream())
    assert good.tolist() == [1, 1]
    c.record[1], c.record[5] = list(c.record[2]), list(c.record[0])
    drafted([1, 2, 5, 0], 9, 4)                                          # twins go on by themselves
    causal([1, 2, 5, 0], 2)
    att.page_free(c.pt, ints([2, 4]), 2, stream())
    c.record[2], c.record[4] = [], []
    used = ints([0])
    att.page_compact(c.pt, c.pt, c.all_maps, used, c.ws, stream())
    assert used.item() == int((c.refs > 0).sum())
    causal([5, 1, 0], 1)
    causal([3, 2], 30)
    drafted([5, 3], 40, 8)
    causal([0, 1, 2, 3, 5], 1)
    for r in (0, 1, 2, 3, 5):                                            # what the rows hold, read back
        n = len(c.record[r])
        k, v = (torch.empty((n, kv, dim), dtype=torch.float32, device="cuda") for _ in "kv")
        att.kv8_read(fmt, *c.maps, c.pt, ints([r] * n), ints(np.arange(n)), tensor_map(k, "f32"), tensor_map(v, "f32"),
                     stream())
        for x, got in enumerate((k, v)):
            assert np.array_equal(f64(got), np.stack([t[x] for t in c.record[r]]))
    att.tile_device_status(stream())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,window,sinks", [("int8", 40, 3), ("e4m3", 25, 2)])
def test_what_is_wrong_is_outside_of_the_limits(fmt, window, sinks, dtype):
    """(No GPU.)  A result of 0, the other head's values, values one token on, a window one short and missing sinks."""
    g = np.random.default_rng(5)
    n, heads, kv, dim, scale = 130, 4, 2, 64, 1 / 8
    q = g.standard_normal((13, heads, dim))
    k, v = g.standard_normal((n, kv, dim)), g.standard_normal((n, kv, dim))
    k, v = (ok.codes(x, ok.code_scale(x, fmt), fmt) * ok.code_scale(x, fmt)[..., None] for x in (k, v))
    sees = ok.causal_sees(n, 13, window, sinks)
    want, limit, lse, near = limits(dtype, q, k, v, sees, scale)
    short, none = ok.causal_sees(n, 13, window - 1, sinks), ok.causal_sees(n, 13, window, 0)
    wrong = {"zero": 0 * want, "heads": ok.attend(q, k, v[:, ::-1], sees, scale)[0],
             "shifted": ok.attend(q, k, np.roll(v, 1, 0), sees, scale)[0],
             "short": ok.attend(q, k, v, short, scale)[0], "none": ok.attend(q, k, v, none, scale)[0]}
    share = {name: (np.abs(x - want) > limit).mean() for name, x in wrong.items()}
    assert all(s > 0.5 for s in share.values()), share
    rows = {name: (np.abs(x - want) > limit).any(-1).all() for name, x in wrong.items()}
    assert all(rows.values()), rows                                      # every query's result, not only some
    for sees in (short, none):
        assert (np.abs(ok.attend(q, k, v, sees, scale)[1] - lse) > near).all()
