"""The failure path of the tcgen05 chunk kernel, made to run on purpose and without
any fault: under PKV_DECODE_TEST_WITHHOLD its producer issues no copy and each
wait is limited to 1 ms, so the first wait for a copy runs out while nothing is
in flight.  The call returns promptly, the status word holds PKV_DEV_TIMEOUT and
nothing else, every row with a key is NaN -- of items written directly, of split
items and of items cut over CTAs, through the merge -- and the next ordinary call
is right with a clean status word."""
from __future__ import annotations

import time

import pytest
import torch

from tests import _chunk
from tests.test_gpu_chunk import pkv  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

# (stored before, new): one key tile; halves of split items; pair items; one item cut
# over every CTA; a mix, items in a row among it
MIXES = {
    "direct": [(5, 1), (0, 100), (90, 7)],
    "split": [(300, 1), (700, 9), (1500, 20)],
    "pair": [(0, 200), (128, 128)],
    "cut": [(20000, 20)],
    "mix": [((i * 53) % 420, 1 + (i % 11 == 0) * (i % 30)) for i in range(120)] + [(9000, 300)],
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (128, True)])
def test_wait_that_runs_out(pkv, mix, d, e4m3):  # noqa: F811
    case = _chunk.make(71, MIXES[mix], 8, 2, d, 16, e4m3=e4m3)
    assert pkv.device_status(reset=True) == 0
    assert pkv.lib.pkv_test_enable_withhold(1) == 0
    try:
        t0 = time.perf_counter()
        out, lse = _chunk.run(pkv, case, flags=pkv.DECODE_TEST_WITHHOLD)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        pkv.lib.pkv_test_enable_withhold(0)
    assert elapsed < 10.0
    assert pkv.device_status(reset=True) == pkv.DEV_TIMEOUT
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse = _chunk.run(pkv, case)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == 0
    _chunk.check(case, out, lse)


def test_control_is_refused_when_not_enabled(pkv):  # noqa: F811
    case = _chunk.make(72, [(5, 3)], 8, 2, 128, 16)
    with pytest.raises(pkv.PkvError):
        _chunk.run(pkv, case, flags=pkv.DECODE_TEST_WITHHOLD)
