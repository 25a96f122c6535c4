"""Values of codes near the largest numbers of f16: the code times the power of two in
its scale is what the product takes, and the rest of the scale goes to the weight."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import require_native  # noqa: E402
from test_gpu_attn_cache import FAR, Setup  # noqa: E402
from test_gpu_attn_cache_edges import set_value_scales  # noqa: E402
from test_gpu_kvcache import gen  # noqa: E402

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_native()


@pytest.mark.parametrize("q_len,hint", [(1, None), (90, FAR)])
@pytest.mark.parametrize("fmt,scale", [("int8", 1000.0), ("e4m3", 4064.0)])
def test_values_beyond_f16_whose_mean_is_not(fmt, scale, q_len, hint):
    """127 * 1000 and 30 * 4064 are above 65504, 127 * 512 and 30 * 2048 are not: the results are as exact as ever,
    where the weights spread so far over the keys (a scale of 1 / 200) that f16 holds them."""
    s = Setup(gen(820), "f16", fmt, [300, 170], None, q_len, 4, 2, 64, 16)
    if fmt == "e4m3":                                                    # codes of 32 and above, halved
        s.v[:, :s.slots] = torch.where(s.v[:, :s.slots] & 0x7F >= 0x60, s.v[:, :s.slots] - 8, s.v[:, :s.slots])
    set_value_scales(s, torch.full((s.pages, 2, 16), scale))
    largest = max(np.abs(s.tokens(s.v, b)).max() for b in (0, 1))
    assert largest > 65504
    got, _ = s.check(0, 0, scale=1 / 200, hint=hint)
    assert np.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,code,scale", [("int8", 127, 1000.0), ("int8", 127, 1024.0), ("e4m3", 0x6C, 1000.0),
                                            ("e4m3", 0x7E, 256.0)])
def test_two_keys_of_equal_weight(fmt, code, scale, dtype):
    """One value of `code` times `scale` beside one of 0.  127 * 1000 and 96 * 1000 stand with 512 times their code,
    which f16 holds: half of the value.  127 * 1024 and 448 * 256 do not: an infinity, though half of them would fit."""
    s = Setup(gen(821), dtype, fmt, [2], None, 1, 2, 1, 64, 16)
    s.q.zero_()
    page = int(s.table[s.rows[0], 0])
    s.v[page, :2] = 0
    s.v[page, 0, 0, ::3] = code
    set_value_scales(s, torch.full((s.pages, 1, 16), scale))
    value = s.tokens(s.v, 0)[0, 0] / 2
    got = s.run()[0][0, 0]
    beyond = dtype == "f16" and scale != 1000.0
    want = np.where(value != 0, np.inf, 0.0) if beyond else value
    step = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    assert value.max() > 40000 and np.array_equal(np.isinf(got), np.tile(np.isinf(want), (2, 1)))
    finite = np.isfinite(want)
    assert (np.abs(got[:, finite] - want[finite]) <= 2 * step * want[finite]).all()   # the weight's rounding, the result's
