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
