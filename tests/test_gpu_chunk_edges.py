"""Chunk attention: buffers a call brings or does not, and inputs at the ends
of what its number formats hold."""
from __future__ import annotations

import pytest
import torch

from tests import _chunk
from tests.test_gpu_chunk import pkv  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def test_small_workspaces_on_two_streams(pkv):  # noqa: F811
    """Calls on a stream of the caller's and on the current one, each with a
    workspace that is too small: neither meets the other's."""
    cases = [_chunk.make(s, [(3000, 200), (700, 1), (0, 90)], 8, 2, 128, 16) for s in (61, 62)]
    want = [_chunk.run(pkv, c)[0] for c in cases]
    bufs = [{n: getattr(c, n).cuda() for n in ("q", "cu", "k_pool", "v_pool", "tables", "lens")}
            for c in cases]
    outs = [(torch.empty_like(w), torch.empty(w.shape[:2], device="cuda")) for w in want]
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for (out, lse), d, c, s in zip(outs, bufs, cases, (side, None)):
            pkv.paged_chunk_attn(d["q"], d["cu"], d["k_pool"], d["v_pool"], d["tables"], d["lens"],
                                 c.scale, workspace=small, out=out, lse=lse, stream=s)
    torch.cuda.synchronize()
    for (out, _), w in zip(outs, want):
        assert torch.equal(out, w)
