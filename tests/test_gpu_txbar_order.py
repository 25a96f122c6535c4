"""The byte-counted barrier's self-test, launched many times: eight copies that
land together report the states that the barrier went through."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import async_tensor_tile_amd as att  # noqa: E402
import oracle  # noqa: E402
import synthgen  # noqa: E402

from gpu_util import empty_dev, encode, require_native, stream, to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu

LAUNCHES, NTILE = 200, 8


@pytest.fixture(scope="module")
def traces():
    """Trace records [LAUNCHES, 2 + NTILE, 4] and the images of the last launch."""
    require_native()
    src = synthgen.u16_bits(11, (128, 64))
    sd = to_dev(src)
    m = encode(sd, "bf16", (64, 128), (128,), (64, 16), swizzle="128b")
    coords = to_dev(np.array([[0, 16 * t] for t in range(NTILE)], dtype=np.int32))
    size = 4 * 4 * (2 + NTILE)
    trace = empty_dev(LAUNCHES * size, 0xFF)
    out = empty_dev(NTILE * 2048, 0)
    for i in range(LAUNCHES):
        att.txbar_selftest(m, coords, NTILE, trace[i * size:], out, stream())
    return to_host(trace).view(np.int32).reshape(LAUNCHES, 2 + NTILE, 4)


def states():
    """(arrivals_left, pending, phase) after each completion, from the oracle's barrier."""
    ob = oracle.Txbar(1)
    ob.arrive_expect_tx(2048 * NTILE)
    want = []
    for _ in range(NTILE):
        ob.complete_tx(2048)
        want.append(ob.state())
    return want


def test_completions_report_their_own_state(traces):
    """An operation that leaves bytes pending reports the phase that it worked
    on, also where the others complete that phase right behind it."""
    for rec in traces:
        got = sorted((tuple(int(x) for x in r[1:]) for r in rec[2:]), key=lambda s: -s[1])
        assert got == sorted(states(), key=lambda s: -s[1])
        assert sorted(rec[2:, 0].tolist()) == list(range(NTILE))


def test_records_stand_in_the_order_of_the_operations(traces):
    for rec in traces:
        assert [tuple(int(x) for x in r[1:]) for r in rec[2:]] == states()
