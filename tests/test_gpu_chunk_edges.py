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


def weigh(case, out, lse, vanish):
    """out and lse against the definition, element by element: the bounds of
    _chunk.check with `vanish` the most that a probability however small is off
    by, as a part of its row's largest."""
    ref, ref_lse, absv, mag, low, qlow = _chunk.reference(case)
    out, lse = out.cpu().double(), lse.cpu().double()
    score = (case.q.shape[2] + 2) * 2.0 ** -24 * mag + 2.0 ** -17 + 2.0 ** -17 * qlow
    assert torch.all((lse - ref_lse).abs() <= score)
    tol = (2.0 ** -11 + 2 * score[..., None]) * absv + 2.0 ** -8 * ref.abs() + vanish * low
    d = (out - ref).abs()
    assert torch.all(d <= tol), float((d / tol).max())


@pytest.mark.parametrize("gap", [12, 14, 16, 18, 20])
@pytest.mark.parametrize("first", [0, 300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 320)])
def test_fp8_long_tail_behind_one_key(pkv, gap, first, window, sinks):  # noqa: F811
    """One key, whose value is 0, takes nearly all of every row: what comes out is
    what the keys `gap` nats below it give.  Their probabilities are fp16 numbers
    2^8 times as large as against the row's largest, off by half a step of 2^-24
    at most: 2^-33 of the largest.  (Against a reference that the largest equals
    they would be off by 2^-25 of it, and vanish 17.4 nats below.)"""
    case = _chunk.make(63, [(1000, 40), (3000, 1)], 8, 2, 128, 16, window=window, sinks=sinks,
                       e4m3=True)
    top = 448 * case.k_scale.double()
    case.k_pool[..., 0] = 0
    for b in range(2):
        rows = (case.tables[b, first // 16].long(), slice(None), first % 16)
        case.k_pool[rows] = 0
        case.k_pool[rows[0], :, rows[2], 0] = 0x7e          # 448
        case.v_pool[rows] = 0
    for h in range(8):
        case.q[:, h, 0] = gap / case.scale / top[h // 4]
    out, lse = _chunk.run(pkv, case)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == 0
    weigh(case, out, lse, 2.0 ** -33)


@pytest.mark.parametrize("k_scale", [1e-2, 1e-8, 1e-30])
def test_fp8_small_queries_over_small_keys(pkv, k_scale):  # noqa: F811
    """Rows of zeros and of the smallest numbers over a head with a small scale:
    all scores are 0 in binary32, the rows are the mean of the values they see."""
    case = _chunk.make(64, [(300, 20), (0, 9)], 8, 2, 128, 16, e4m3=True)
    case.k_scale[:] = k_scale
    case.q[::3] = 0
    case.q[1::3] *= 2.0 ** -120
    out, lse = _chunk.run(pkv, case)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == 0
    _chunk.check(case, out, lse)
    weigh(case, out, lse, 2.0 ** -24)


@pytest.mark.parametrize("e4m3", [False, True])
def test_cuda_core_rows_that_are_not_numbers(pkv, e4m3):  # noqa: F811
    """A NaN in a query or in a key a row sees: that row is NaN in the CUDA-core
    form too, also where it has no other score."""
    case = _chunk.make(65, [(300, 20), (0, 3)], 8, 2, 128, 16, e4m3=e4m3)
    want = _chunk.run(pkv, case, flags=pkv.DECODE_GENERIC)
    case.q[7, 5, 3] = float("nan")
    case.q[20, 1, 0] = float("nan")         # sees one key
    out, lse = _chunk.run(pkv, case, flags=pkv.DECODE_GENERIC)
    torch.cuda.synchronize()
    rest = torch.ones(out.shape[:2], dtype=torch.bool)
    for t, h in ((7, 5), (20, 1)):
        assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h])
        rest[t, h] = False
    assert torch.equal(out[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])
    # every key of the second sequence's first row, which is its only one
    case.k_pool[case.tables[1, 0].long(), :, 0] = 0x7f if e4m3 else float("nan")
    out, lse = _chunk.run(pkv, case, flags=pkv.DECODE_GENERIC)
    torch.cuda.synchronize()
    assert torch.isnan(out[20]).all() and torch.isnan(lse[20]).all()
    assert pkv.device_status(reset=True) == 0


def test_workspaces_on_the_host_or_with_gaps_are_refused(pkv):  # noqa: F811
    case = _chunk.make(66, [(300, 20)], 8, 2, 128, 16)
    with pytest.raises(TypeError):
        _chunk.run(pkv, case, workspace=torch.empty(1 << 26, dtype=torch.uint8))
    with pytest.raises(ValueError):
        _chunk.run(pkv, case, workspace=torch.empty(1 << 27, dtype=torch.uint8, device="cuda")[::2])
    assert pkv.device_status(reset=True) == 0


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("length", [-1, -2 ** 31, 65, 2 ** 31 - 1])
def test_bad_length_of_a_sequence_without_new_tokens(pkv, flags, length):  # noqa: F811
    """It sets the status as any other does, in both forms, and changes no row."""
    case = _chunk.make(67, [(30, 4), (50, 0), (0, 9)], 8, 2, 128, 16)
    assert case.tables.shape[1] == 4
    case.lens[1] = length
    out, lse = _chunk.run(pkv, case, flags=flags)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == pkv.DEV_SEQ_LEN
    _chunk.check(case, out, lse)
