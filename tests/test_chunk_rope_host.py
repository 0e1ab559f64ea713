"""Host checks of the chunk attention and rope_append calls, the frequency
table, and the binding's own checks: nothing here reaches a GPU."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    return m


P, BAD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


def chunk(pkv, desc=(16, 16, 8, 128, 128), q=P, T=4, hq=32, cu=P, batch=2, k=P, v=P, tables=P,
          max_blocks=4, lens=P, scale=1.0, window=0, sinks=0, ws=None, nbytes=0, out=P, lse=P,
          flags=0):
    d = pkv.CacheDesc(*desc)
    return pkv.lib.pkv_paged_chunk_attn(ctypes.byref(d), q, T, hq, cu, batch, k, v, tables,
                                        max_blocks, lens, scale, window, sinks, ws, nbytes, out,
                                        lse, flags, None)


def chunk_e4m3(pkv, desc=(16, 16, 8, 128, 128), v=P, ks=P, vs=P, T=4, scale=1.0):
    d = pkv.CacheDesc(*desc)
    return pkv.lib.pkv_paged_chunk_attn_e4m3(ctypes.byref(d), P, T, 32, P, 2, P, v, ks, vs, P, 4,
                                             P, scale, 0, 0, None, 0, P, P, 0, None)


def test_chunk_refusals(pkv):
    for name in ("q", "cu", "k", "tables", "lens", "out"):
        assert chunk(pkv, **{name: None}) == -1, name
    for name in ("q", "k", "v", "out"):
        assert chunk(pkv, **{name: BAD}) == -3, name
    for kw in (dict(T=-1), dict(batch=-1), dict(hq=0), dict(max_blocks=-1), dict(window=-1),
               dict(sinks=-1), dict(flags=4), dict(flags=0x100)):
        assert chunk(pkv, **kw) == -1, kw
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert chunk(pkv, scale=scale) == -1
    for desc in ((0, 16, 8, 128, 128), (16, 0, 8, 128, 128), (16, 257, 8, 128, 128),
                 (16, 16, 0, 128, 128)):
        assert chunk(pkv, desc=desc) == -1
    for desc in ((16, 16, 8, 100, 128), (16, 16, 8, 128, 1032), (16, 16, 5, 128, 128)):
        assert chunk(pkv, desc=desc) == -2
    assert chunk(pkv, desc=(16, 16, 8, 64, 128), v=None) == -2
    assert chunk(pkv, batch=65536) == -2
    assert chunk(pkv, T=1 << 27) == -2            # 2^32 rows
    # nothing to do is a success that launches nothing
    assert chunk(pkv, T=0, q=None) == 0 and chunk(pkv, batch=0, cu=None) == 0
    assert chunk_e4m3(pkv, v=None) == -1
    assert chunk_e4m3(pkv, scale=0.0) == -1


def test_chunk_workspace_is_checked(pkv):
    desc = pkv.CacheDesc(16, 16, 8, 128, 128)
    need = pkv.lib.pkv_chunk_workspace_size(ctypes.byref(desc), 4, 2, 32, 4, 0)
    if need:
        assert chunk(pkv) == -4
        assert chunk(pkv, ws=P, nbytes=need - 1) == -4
        assert chunk(pkv, ws=BAD, nbytes=need) == -3
    # the CUDA-core form needs none; refused shapes have none
    assert pkv.lib.pkv_chunk_workspace_size(ctypes.byref(desc), 4, 2, 32, 4, 1) == 0
    assert pkv.lib.pkv_chunk_workspace_size(ctypes.byref(desc), -1, 2, 32, 4, 0) == 0
    assert pkv.lib.pkv_chunk_workspace_size(ctypes.byref(desc), 4, 2, 0, 4, 0) == 0
    assert pkv.lib.pkv_chunk_workspace_size(None, 4, 2, 32, 4, 0) == 0


def rope(pkv, desc=(16, 16, 8, 128, 128), k=P, v=P, q=P, hq=32, kn=P, vn=P, pos=P, slots=P, T=4,
         inv=P, rot=128, off=0, amp=1.0, flags=0, out=ctypes.c_void_p(0x2000)):
    d = pkv.CacheDesc(*desc)
    return pkv.lib.pkv_rope_append(ctypes.byref(d), k, v, q, hq, kn, vn, pos, slots, T, inv, rot,
                                   off, amp, flags, out, None)


def test_rope_refusals(pkv):
    for name in ("q", "kn", "k", "pos", "slots", "inv", "out", "v", "vn"):
        assert rope(pkv, **{name: None}) == -1, name
    for name in ("q", "kn", "k", "v", "vn", "out"):
        assert rope(pkv, **{name: BAD}) == -3, name
    for kw in (dict(rot=0), dict(rot=3), dict(rot=130), dict(off=-1), dict(rot=64, off=65),
               dict(hq=4090)):
        assert rope(pkv, **kw) == -2, kw
    for kw in (dict(T=-1), dict(hq=0), dict(flags=4), dict(amp=math.inf), dict(amp=math.nan),
               dict(flags=2, out=P)):             # fp32 cannot overwrite bf16
        assert rope(pkv, **kw) == -1, kw
    assert rope(pkv, desc=(16, 16, 8, 100, 128)) == -1
    assert rope(pkv, desc=(16, 16, 8, 64, 128), v=None, vn=None, rot=64) == -2
    assert rope(pkv, T=0, q=None) == 0
    d = pkv.CacheDesc(16, 16, 8, 128, 128)
    call = pkv.lib.pkv_rope_append_e4m3
    o = ctypes.c_void_p(0x2000)
    args = lambda v, vn, ks, vs: (ctypes.byref(d), P, v, P, 32, P, vn, ks, vs, P, P, 4, P, 128, 0,
                                  1.0, 0, o, None)
    assert call(*args(None, None, P, P)) == -1
    assert call(*args(ctypes.c_void_p(0x1004), P, P, P)) == -3


def test_frequencies(pkv):
    f = pkv.rope_frequencies(128, device="cpu")
    i = torch.arange(64, dtype=torch.float64)
    plain = 10000.0 ** (-2 * i / 128)
    assert torch.allclose(f, plain, rtol=1e-14, atol=0)
    assert torch.allclose(pkv.rope_frequencies(128, factor=8.0, device="cpu"), plain / 8,
                          rtol=1e-14, atol=0)
    theta, factor, ctx, low, high = 500000.0, 8.0, 8192, 1.0, 4.0
    f = pkv.rope_frequencies(128, theta, factor, ctx, low, high, device="cpu")
    base = theta ** (-2 * i / 128)
    turns = ctx * base / (2 * math.pi)
    for j in range(64):
        if turns[j] >= high:
            want = base[j]
        elif turns[j] <= low:
            want = base[j] / factor
        else:
            keep = (turns[j] - low) / (high - low)
            want = keep * base[j] + (1 - keep) * base[j] / factor
        assert abs(f[j] - want) <= 1e-14 * want
    assert (turns >= high).any() and (turns <= low).any()


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=5), dict(theta=0.0),
                                dict(theta=math.inf), dict(factor=0.5), dict(factor=math.nan),
                                dict(original_len=-1), dict(original_len=64, low_turns=0.0),
                                dict(original_len=64, low_turns=4.0, high_turns=4.0)])
def test_frequencies_refused(pkv, kw):
    with pytest.raises(pkv.PkvError):
        pkv.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})


def test_binding_refuses_cpu_tensors_and_other_types(pkv):
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.paged_chunk_attn(q, i32, pool, pool, i32.view(1, 2), i32[:1], 1.0)
    with pytest.raises(TypeError):
        pkv.rope_append(pool, pool, q, q, q, i32, i32, torch.zeros(64))
