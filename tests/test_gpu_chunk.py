"""Attention of ragged chunks of new tokens over the paged cache
(pkv_paged_chunk_attn and its E4M3 form) against the definition in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests import _chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    m.device_status(reset=True)
    return m


def both(pkv, case, flags=0, status=0):
    out, lse = _chunk.run(pkv, case, flags=flags)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == status
    _chunk.check(case, out, lse)
    return out, lse


# (stored before, new) of each sequence
MIXES = {
    "one": [(0, 1)],
    "first": [(0, 37)],
    "tiles": [(0, 256), (128, 128), (127, 129)],
    "ragged": [(5, 1), (0, 3), (300, 70), (17, 0), (1, 200), (255, 1)],
    "long": [(511, 33), (1000, 1)],
}


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (8, 1, 64, 32), (4, 4, 128, 8),
                                   (14, 2, 128, 64), (16, 1, 64, 256)])
def test_dense(pkv, mix, shape):
    hq, hkv, d, bs = shape
    both(pkv, _chunk.make(1, MIXES[mix], hq, hkv, d, bs, poison=True))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (100, 0), (128, 1), (129, 130),
                                          (300, 64), (5000, 4)])
@pytest.mark.parametrize("mix", ["ragged", "long", "tiles"])
def test_window_and_sinks(pkv, mix, window, sinks):
    both(pkv, _chunk.make(2, MIXES[mix], 8, 2, 128, 16, window=window, sinks=sinks, poison=True))


@pytest.mark.parametrize("window,sinks", [(40, 5), (700, 0)])
def test_window_small_heads(pkv, window, sinks):
    both(pkv, _chunk.make(3, MIXES["ragged"] + [(900, 300)], 16, 2, 64, 64, window=window,
                          sinks=sinks, poison=True))


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4), (300, 0)])
@pytest.mark.parametrize("shape", [(8, 2, 16), (8, 1, 32), (16, 1, 128), (6, 2, 64)])
def test_e4m3(pkv, shape, window, sinks):
    hq, hkv, bs = shape
    both(pkv, _chunk.make(4, MIXES["ragged"] + [(400, 150)], hq, hkv, 128, bs, window=window,
                          sinks=sinks, e4m3=True, poison=True))


# shapes of no tensor-core tile: odd head dims, block sizes, values inside the keys
@pytest.mark.parametrize("kw", [
    dict(hq=6, hkv=2, dk=72, bs=5), dict(hq=4, hkv=4, dk=8, bs=1), dict(hq=3, hkv=1, dk=128, bs=48),
    dict(hq=8, hkv=1, dk=192, dv=128, bs=16), dict(hq=16, hkv=1, dk=576, dv=512, bs=64, latent=True),
    dict(hq=2, hkv=2, dk=1024, bs=16), dict(hq=8, hkv=2, dk=96, bs=16, e4m3=True),
    dict(hq=160, hkv=1, dk=64, bs=16),
], ids=str)
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4)])
def test_generic_shapes(pkv, kw, window, sinks):
    both(pkv, _chunk.make(5, [(5, 1), (0, 3), (100, 20), (17, 0)], window=window, sinks=sinks,
                          poison=True, **kw))


@pytest.mark.parametrize("e4m3", [False, True])
def test_generic_flag(pkv, e4m3):
    case = _chunk.make(6, MIXES["ragged"], 8, 2, 128, 16, e4m3=e4m3)
    both(pkv, case, flags=pkv.DECODE_GENERIC)
    both(pkv, case, flags=pkv.DECODE_NO_TCGEN05)


@pytest.mark.parametrize("e4m3", [False, True])
def test_padding_rows_are_left(pkv, e4m3):
    case = _chunk.make(7, [(10, 5), (0, 0), (0, 130)], 8, 2, 128, 16, pad=(3, 140), e4m3=e4m3)
    T = case.q.shape[0]
    out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 8), 7.0, device="cuda")
    _chunk.run(pkv, case, out=out, lse=lse)
    torch.cuda.synchronize()
    for t in (out, lse):
        assert torch.all(t[:3] == 7) and torch.all(t[T - 140:] == 7)
    _chunk.check(case, out, lse)


@pytest.mark.parametrize("flags", [0, 1])
def test_fewer_stored_than_new(pkv, flags):
    """seq_len 0, and 2 stored of 5 new: the rows without a token are empty."""
    case = _chunk.make(8, [(0, 4), (0, 5), (40, 3)], 8, 2, 128, 16)
    case.lens[0], case.lens[1] = 0, 2
    both(pkv, case, flags=flags, status=pkv.DEV_SEQ_LEN)


@pytest.mark.parametrize("flags", [0, 1])
def test_seq_len_past_its_table(pkv, flags):
    case = _chunk.make(9, [(0, 4), (60, 3)], 8, 2, 128, 16)
    good = case.lens.clone()
    case.lens[1] = case.tables.shape[1] * 16 + 1
    out, lse = _chunk.run(pkv, case, flags=flags)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) == pkv.DEV_SEQ_LEN
    assert torch.all(out[4:] == 0) and torch.all(torch.isinf(lse[4:]))
    case.lens = good
    both(pkv, case, flags=flags)


@pytest.mark.parametrize("flags", [0, 1])
def test_bad_table_entry(pkv, flags):
    case = _chunk.make(10, [(0, 20), (60, 3)], 8, 2, 128, 16)
    good = case.tables.clone()
    for bad in (-1, case.k_pool.shape[0], 2 ** 31 - 1):
        case.tables = good.clone()
        case.tables[1, 1] = bad
        out, lse = _chunk.run(pkv, case, flags=flags)
        torch.cuda.synchronize()
        assert pkv.device_status(reset=True) == pkv.DEV_BLOCK_ID
        case.tables = good
        ref = _chunk.reference(case)[1]
        assert torch.allclose(lse[:20].cpu().double(), ref[:20], atol=1e-3)


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("cu", [[0, 9, 4, 20], [0, 5, 10, 21], [-1, 5, 10, 20], [0, 30, 40, 20],
                                [2 ** 31 - 1] * 4, [0, -2 ** 31, 2 ** 31 - 1, 20]])
def test_bad_cu_q_lens(pkv, cu, flags):
    case = _chunk.make(11, [(0, 5), (7, 5), (60, 10)], 8, 2, 128, 16)
    case.cu = torch.tensor(cu, dtype=torch.int32)
    _chunk.run(pkv, case, flags=flags)
    torch.cuda.synchronize()
    assert pkv.device_status(reset=True) & pkv.DEV_QUERY_RANGE


def test_large_scores_and_scale(pkv):
    """Scores of some hundreds: one key takes nearly everything."""
    case = _chunk.make(12, [(200, 60), (3, 1)], 8, 2, 128, 16, scale=3.0)
    both(pkv, case)
    case = _chunk.make(12, [(200, 60), (3, 1)], 8, 2, 128, 16, scale=1e-6)
    both(pkv, case)


def test_rising_and_falling_scores(pkv):
    """The running maximum rises at every tile, or only at the first."""
    for up in (False, True):
        case = _chunk.make(13, [(900, 100)], 4, 1, 128, 16)
        L = 1000
        ramp = torch.linspace(0, 40, L) if up else torch.linspace(40, 0, L)
        case.q[:] = 0
        case.q[:, :, 0] = math.sqrt(128)
        j = torch.arange(L)
        case.k_pool[case.tables[0, j // 16].long(), 0, j % 16, 0] = ramp.to(torch.bfloat16)
        both(pkv, case)


def test_many_sequences(pkv):
    """More sequences than any table of the kernel's plan holds at once."""
    chunks = [((i * 37) % 90, 1 + (i % 3 == 0) * (i % 7)) for i in range(1500)]
    both(pkv, _chunk.make(14, chunks, 4, 2, 64, 16))


def test_bf16_zero_batch(pkv):
    case = _chunk.make(15, [(3, 2)], 8, 2, 128, 16)
    dev = "cuda"
    out, lse = pkv.paged_chunk_attn(case.q.to(dev)[:0], torch.zeros(1, dtype=torch.int32, device=dev),
                                    case.k_pool.to(dev), case.v_pool.to(dev),
                                    case.tables.to(dev)[:0], case.lens.to(dev)[:0], 1.0)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


def _fixed(case, pkv, dev="cuda"):
    """Device buffers of one call, for captures and repeats."""
    t = {n: getattr(case, n).to(dev) for n in ("q", "cu", "k_pool", "v_pool", "tables", "lens")}
    T, hq, _ = case.q.shape
    t["out"] = torch.empty(T, hq, case.dv, dtype=torch.bfloat16, device=dev)
    t["lse"] = torch.empty(T, hq, device=dev)
    need = pkv.chunk_workspace_size(t["k_pool"], t["v_pool"], T, case.lens.numel(), hq,
                                    case.tables.shape[1])
    t["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=dev)

    def call(stream=None):
        pkv.paged_chunk_attn(t["q"], t["cu"], t["k_pool"], t["v_pool"], t["tables"], t["lens"],
                             case.scale, window=case.window, sink_tokens=case.sinks,
                             workspace=t["ws"], out=t["out"], lse=t["lse"], stream=stream)
    return t, call


@pytest.mark.parametrize("mix", ["ragged", "long"])
def test_repeated_calls_return_identical_bits(pkv, mix):
    case = _chunk.make(16, MIXES[mix] + [(2000, 300)], 8, 2, 128, 16)
    t, call = _fixed(case, pkv)
    call()
    torch.cuda.synchronize()
    out, lse = t["out"].clone(), t["lse"].clone()
    for _ in range(50):
        t["out"].fill_(3)
        t["ws"].fill_(255)
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, t["out"]) and torch.equal(lse, t["lse"])
    _chunk.check(case, out, lse)


def test_graph_replay_with_new_lengths(pkv):
    """One capture serves other lengths and chunk boundaries of the same sizes."""
    a = _chunk.make(17, [(100, 40), (0, 24), (700, 1)], 8, 2, 128, 16, window=200, sinks=4)
    t, call = _fixed(a, pkv)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b = _chunk.make(18, [(3, 1), (500, 63), (40, 1)], 8, 2, 128, 16, window=200, sinks=4)
    for case in (a, b, a):
        for n in ("q", "cu", "lens"):
            t[n].copy_(getattr(case, n))
        t["tables"].fill_(-1)
        t["tables"][:, :case.tables.shape[1]].copy_(case.tables)
        t["k_pool"][:case.k_pool.shape[0]].copy_(case.k_pool)
        t["v_pool"][:case.v_pool.shape[0]].copy_(case.v_pool)
        graph.replay()
        torch.cuda.synchronize()
        _chunk.check(case, t["out"], t["lse"])
    assert pkv.device_status(reset=True) == 0


def test_two_streams_at_once(pkv):
    cases = [_chunk.make(s, MIXES["ragged"] + [(1500, 200)], 8, 2, 128, 16) for s in (19, 20)]
    bufs = [_fixed(c, pkv) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (t, call), s in zip(bufs, streams):
            call(stream=s)
    torch.cuda.synchronize()
    for c, (t, _) in zip(cases, bufs):
        _chunk.check(c, t["out"], t["lse"])


def test_lse_not_wanted(pkv):
    """The C call without an LSE buffer."""
    import ctypes
    case = _chunk.make(21, MIXES["ragged"], 8, 2, 128, 16)
    t, call = _fixed(case, pkv)
    call()
    torch.cuda.synchronize()
    want = t["out"].clone()
    t["out"].fill_(0)
    p = lambda x: ctypes.c_void_p(x.data_ptr())
    desc = pkv.cache_desc(t["k_pool"], t["v_pool"])
    rc = pkv.lib.pkv_paged_chunk_attn(
        ctypes.byref(desc), p(t["q"]), case.q.shape[0], 8, p(t["cu"]), case.lens.numel(),
        p(t["k_pool"]), p(t["v_pool"]), p(t["tables"]), case.tables.shape[1], p(t["lens"]),
        case.scale, 0, 0, p(t["ws"]), t["ws"].numel(), p(t["out"]), None, 0,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(want, t["out"])


def test_agrees_with_decode_and_multi(pkv):
    """Single tokens: the decode attention's result; T tokens per sequence: the
    multi-token call's (both take fp32 queries and return fp32)."""
    for T in (1, 4):
        case = _chunk.make(22, [(300, T), (17, T), (64, T)], 32, 8, 128, 16)
        dev = "cuda"
        out, lse = _chunk.run(pkv, case)
        k, v = case.k_pool.to(dev), case.v_pool.to(dev)
        q = case.q.to(dev).float().view(3, T, 32, 128)
        ro, rl = pkv.paged_decode_attn_multi(q, k, v, case.tables.to(dev), case.lens.to(dev),
                                             case.scale)
        assert torch.allclose(lse, rl.view(3 * T, 32), atol=1e-4)
        assert torch.allclose(out.float(), ro.view(3 * T, 32, 128), atol=2e-2)
