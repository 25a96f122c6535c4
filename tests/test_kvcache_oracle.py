"""The oracle's attention for long prefixes against the one written key by key."""
import numpy as np
import pytest

from oracle import kvcache as ok


@pytest.mark.parametrize("prefix, lens, q_len", [(0, [3, 0, 7], 1), (9, [2, 5, 0], 3), (20, [0, 11, 4], 2)])
def test_attention_by_head(prefix, lens, q_len):
    rng = np.random.default_rng(prefix)
    q = rng.standard_normal((3, q_len, 4, 8))
    k, v = (rng.standard_normal((12, 4, 2, 8)) for _ in "kv")
    table = rng.permutation(np.tile(np.arange(12), 2))[:20].reshape(4, 5)
    rows, full = [3, 0, 2], np.zeros(4, dtype=int)
    full[rows] = lens
    full[1] = prefix
    args = (q, k, v, table, full, 4, 1, prefix, rows, 0.3)
    for a, b in zip(ok.attention(*args), ok.attention_by_head(*args)):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-12)
