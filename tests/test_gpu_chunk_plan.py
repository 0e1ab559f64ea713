"""Chunk attention where its work is cut over the GPU, at the ends of its
arguments' ranges, and in calls that overlap."""
from __future__ import annotations

import math

import pytest
import torch

from tests import _chunk
from tests.test_gpu_chunk import _fixed, both, pkv  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


# (chunks, query heads, KV heads, head dim, block size, window, sinks)
PLANS = {
    # one block of query tokens, its keys cut over every CTA
    "one_pair": ([(20000, 32)], 8, 1, 128, 16, 0, 0),
    "one_token": ([(30000, 1)], 8, 2, 128, 16, 0, 0),
    # both kinds of item, of very uneven lengths
    "uneven": ([(30000, 1), (0, 700), (9, 1), (12000, 130), (0, 0), (2500, 33), (1, 1)], 8, 2,
               128, 16, 0, 0),
    "uneven_small_heads": ([(9000, 1), (0, 500), (3000, 77)], 8, 2, 64, 32, 0, 0),
    # whole rounds and a cut rest, alike blocks (by KV head) and unlike ones
    "alike": ([(1000, 4)] * 90, 8, 4, 128, 16, 0, 0),
    "unlike": ([(200 * i, 20) for i in range(40)], 8, 8, 64, 16, 0, 0),
    "windowed": ([(500 * i + 7, 90) for i in range(14)], 8, 4, 64, 16, 777, 5),
    # more query blocks than are sorted: of many tokens, and of many sequences
    "blocks": ([(3 * i % 50, 17) for i in range(600)], 32, 1, 128, 16, 0, 0),
    "sequences": ([(i % 70, 1 + i % 9) for i in range(1100)], 32, 1, 128, 16, 60, 2),
    # a row tile is one token, and an odd group
    "whole_group": ([(300, 5), (0, 140)], 128, 1, 128, 16, 0, 0),
    "odd_group": ([(300, 5), (0, 140), (2000, 1)], 27, 1, 128, 64, 0, 0),
}


@pytest.mark.parametrize("name", PLANS)
def test_plans(pkv, name):  # noqa: F811
    chunks, hq, hkv, d, bs, window, sinks = PLANS[name]
    both(pkv, _chunk.make(41, chunks, hq, hkv, d, bs, window=window, sinks=sinks, poison=True))


@pytest.mark.parametrize("name", ["one_pair", "one_token", "uneven", "alike", "blocks",
                                  "whole_group"])
def test_plans_e4m3(pkv, name):  # noqa: F811
    chunks, hq, hkv, d, bs, window, sinks = PLANS[name]
    both(pkv, _chunk.make(42, chunks, hq, hkv, d, max(bs, 16), window=window, sinks=sinks,
                          poison=True, e4m3=True))


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1),
                                          (0, 2 ** 31 - 1), (50, 2 ** 31 - 1), (50, 330), (1, 0)])
def test_largest_window_and_sinks(pkv, window, sinks, flags):  # noqa: F811
    case = _chunk.make(43, [(300, 30), (0, 5), (0, 9)], 8, 2, 128, 16, window=window, sinks=sinks)
    case.lens[2] = 4                       # five rows before the first position
    both(pkv, case, flags=flags, status=pkv.DEV_SEQ_LEN)


@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_that_jump_inside_a_tile(pkv, e4m3):  # noqa: F811
    """Each 64 keys' scores lie some tens above or below the 64 before."""
    case = _chunk.make(44, [(1200, 40), (500, 1)], 8, 2, 128, 16, e4m3=e4m3)
    level = torch.tensor([0, 30, 10, 60, 61, 20, 90, 120, 5, 0, 130, 131, 100, 0, 135, 3, 140,
                          20, 139, 160])
    # key channel 0 holds the level (E4M3 codes: 128 and 448 are exact)
    steps = level.double() / 160 * 15
    q0 = 160 / 15 / case.scale
    case.q[..., 0] = q0
    for b, L in enumerate(case.lens.tolist()):
        j = torch.arange(L)
        rows = (case.tables[b, j // 16].long(), j % 16)
        want = steps[j // 64]
        for h in range(2):
            if e4m3:
                code = (want / case.k_scale[h].double()).clamp(-448, 448)
                code = code.float().to(torch.float8_e4m3fn).view(torch.uint8)
                case.k_pool[rows[0], h, rows[1], 0] = code
            else:
                case.k_pool[rows[0], h, rows[1], 0] = want.to(torch.bfloat16)
    both(pkv, case)


def test_large_values(pkv):  # noqa: F811
    """Values up to 2^78 with scores that pass the first by far."""
    case = _chunk.make(45, [(900, 20)], 4, 1, 128, 16)
    case.v_pool *= 2.0 ** 76
    both(pkv, case)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_that_are_not_finite(pkv, bad, e4m3):  # noqa: F811
    """Such a row is NaN and its neighbours are not touched."""
    case = _chunk.make(46, [(300, 20), (40, 1)], 8, 2, 128, 16, e4m3=e4m3)
    want, _ = _chunk.run(pkv, case)
    case.q[7, 5, 3] = bad
    out, lse = _chunk.run(pkv, case)
    torch.cuda.synchronize()
    assert torch.isnan(out[7, 5]).all() and torch.isnan(lse[7, 5])
    rest = torch.ones(out.shape[:2], dtype=torch.bool)
    rest[7, 5] = False
    assert torch.equal(out[rest], want[rest])
    assert pkv.device_status(reset=True) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_queries_of_any_size(pkv, e4m3):  # noqa: F811
    """Rows whose magnitudes span what bf16 spans: scores, not the queries'
    size, are what the E4M3 terms have to hold."""
    case = _chunk.make(47, [(300, 20)], 8, 2, 128, 16, e4m3=e4m3)
    size = 2.0 ** torch.linspace(-120, 3, 20)
    case.q = (case.q.float() * size[:, None, None]).to(torch.bfloat16)
    case.q[4] = 0
    both(pkv, case)


@pytest.mark.parametrize("e4m3", [False, True])
def test_buffers_on_odd_16_byte_boundaries(pkv, e4m3):  # noqa: F811
    case = _chunk.make(48, [(900, 20), (5000, 1), (0, 200)], 8, 2, 128, 16, e4m3=e4m3)
    T = case.q.shape[0]
    want = _chunk.run(pkv, case)
    out = torch.empty(T * 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(T, 8, 128)
    lse = torch.empty(T * 8 + 1, device="cuda")[1:].view(T, 8)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")[16:]
    got = _chunk.run(pkv, case, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_workspace_size_is_enough(pkv):  # noqa: F811
    """Nothing is written past the size that is asked for."""
    for name in ("uneven", "blocks", "sequences", "unlike"):
        chunks, hq, hkv, d, bs, window, sinks = PLANS[name]
        case = _chunk.make(49, chunks, hq, hkv, d, bs, window=window, sinks=sinks)
        need = pkv.chunk_workspace_size(case.k_pool.cuda(), case.v_pool.cuda(), case.q.shape[0],
                                        case.lens.numel(), hq, case.tables.shape[1])
        buf = torch.full((need + 4096 + 16,), 0xa5, dtype=torch.uint8, device="cuda")
        for off in (0, 16):
            _chunk.run(pkv, case, workspace=buf[off:off + need])
            torch.cuda.synchronize()
            assert torch.all(buf[off + need:] == 0xa5) and torch.all(buf[:off] == 0xa5)
            buf.fill_(0xa5)


def test_a_stream_of_ones_own(pkv):  # noqa: F811
    """`stream` other than the current one, buffers made by the call."""
    case = _chunk.make(50, [(900, 20), (5000, 1)], 8, 2, 128, 16)
    want = _chunk.run(pkv, case)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    dev = {n: getattr(case, n).cuda() for n in ("q", "cu", "k_pool", "v_pool", "tables", "lens")}
    torch.cuda.synchronize()
    for _ in range(3):
        got = pkv.paged_chunk_attn(dev["q"], dev["cu"], dev["k_pool"], dev["v_pool"],
                                   dev["tables"], dev["lens"], case.scale, stream=s)
        again = pkv.paged_chunk_attn(dev["q"], dev["cu"], dev["k_pool"], dev["v_pool"],
                                     dev["tables"], dev["lens"], case.scale)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(again[0], want[0])


def test_two_graphs_at_once(pkv):  # noqa: F811
    """Captures that bring no workspace get one each and may run together."""
    cases = [_chunk.make(s, [(3000, 200), (700, 1)], 8, 2, 128, 16) for s in (51, 52)]
    graphs = []
    for c in cases:
        dev = {n: getattr(c, n).cuda() for n in ("q", "cu", "k_pool", "v_pool", "tables", "lens")}
        call = lambda: pkv.paged_chunk_attn(dev["q"], dev["cu"], dev["k_pool"], dev["v_pool"],
                                            dev["tables"], dev["lens"], c.scale)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, dev, out, torch.cuda.Stream()))
    for _ in range(20):
        for g, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (_, _, (out, lse), _) in zip(cases, graphs):
        _chunk.check(c, out, lse)
    assert pkv.device_status(reset=True) == 0


def test_two_threads_on_one_stream(pkv):  # noqa: F811
    """Calls of two threads may interleave kernel by kernel on their stream."""
    import threading
    cases = [_chunk.make(s, [(3000, 200), (700, 1), (0, 90)], 8, 2, 128, 16) for s in (53, 54)]
    want = [_chunk.run(pkv, c)[0] for c in cases]
    bufs = [{n: getattr(c, n).cuda() for n in ("q", "cu", "k_pool", "v_pool", "tables", "lens")}
            for c in cases]
    torch.cuda.synchronize()
    wrong = [0, 0]

    def work(k):
        d = bufs[k]
        for _ in range(200):
            out, _ = pkv.paged_chunk_attn(d["q"], d["cu"], d["k_pool"], d["v_pool"], d["tables"],
                                          d["lens"], cases[k].scale)
            wrong[k] += int(not torch.equal(out, want[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_short_items_in_a_row(pkv, d, e4m3, window, sinks):  # noqa: F811
    """Items of one and of two key tiles, mixed: their second half has nothing to
    do for some items, and must not run ahead of the first."""
    chunks = [((i * 53) % 420, 1 + (i % 11 == 0) * (i % 30)) for i in range(144)]
    case = _chunk.make(55, chunks, 24, 8, d, 16, window=window, sinks=sinks, poison=True, e4m3=e4m3)
    out, lse = both(pkv, case)
    for _ in range(20):
        again = _chunk.run(pkv, case)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
