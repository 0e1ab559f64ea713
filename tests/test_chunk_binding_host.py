"""The chunk attention binding's own work -- buffers, streams, arguments --
without a GPU: CUDA's streams are stood in for, and no library call is made
that would launch."""
from __future__ import annotations

import contextlib
import threading
from types import SimpleNamespace

import pytest
import torch

NEED = 4096


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    return m


@pytest.fixture
def pkv(built, monkeypatch):
    """The binding on CPU tensors; `pkv.now[0]` is the current stream's handle."""
    now, capturing = [0], set()

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s.cuda_stream
        try:
            yield
        finally:
            now[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0] in capturing)
    monkeypatch.setattr(built, "_stream", lambda s=None: now[0] if s is None else s.cuda_stream)
    monkeypatch.setattr(built, "_need", lambda *a, **k: None)
    monkeypatch.setattr(built, "_chunk_scratch", threading.local())
    return SimpleNamespace(m=built, now=now, capturing=capturing)


SIDE = SimpleNamespace(cuda_stream=7)


def scratch(pkv, stream=None, brings="none", outputs=False, need=NEED):
    """The workspace a call uses."""
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    cu, lens = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws = {"none": None, "small": torch.empty(NEED // 2, dtype=torch.uint8),
          "enough": torch.empty(NEED, dtype=torch.uint8)}[brings]
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16) if outputs else None
    lse = torch.empty(3, 8) if outputs else None
    got, size, _, _ = pkv.m._chunk_args(pkv.m.CacheDesc(4, 16, 2, 128, 128), lambda *a: need, q,
                                        cu, torch.zeros(1, 4, dtype=torch.int32), lens, ws, out,
                                        lse, 0, stream)
    assert got.numel() == size >= need
    assert (got is ws) == (brings == "enough")
    return got


@pytest.mark.parametrize("outputs", [False, True])
@pytest.mark.parametrize("here", ["none", "small", "enough"])
@pytest.mark.parametrize("there", ["none", "small", "enough"])
def test_streams_never_share_scratch(pkv, there, here, outputs):
    """A call on a stream of the caller's and one on the current stream may run
    at once, whatever each brings."""
    a = scratch(pkv, SIDE, there, outputs)
    b = scratch(pkv, None, here, outputs)
    assert a.data_ptr() != b.data_ptr()
    # each stream's own is kept, and is the same whichever way the stream is named
    if there != "enough":
        assert scratch(pkv, SIDE, "small", True) is a
        pkv.now[0] = SIDE.cuda_stream
        assert scratch(pkv, None, "none", outputs) is a


@pytest.mark.parametrize("brings", ["none", "small"])
@pytest.mark.parametrize("outputs", [False, True])
def test_a_capture_on_a_side_stream_gets_scratch_of_its_own(pkv, brings, outputs):
    kept = [scratch(pkv), scratch(pkv, SIDE)]
    pkv.capturing.add(SIDE.cuda_stream)
    a, b = (scratch(pkv, SIDE, brings, outputs) for _ in range(2))
    assert len({t.data_ptr() for t in (a, b, *kept)}) == 4
    pkv.capturing.clear()
    assert scratch(pkv) is kept[0] and scratch(pkv, SIDE) is kept[1]


def test_scratch_grows_on_its_own_stream(pkv):
    main, side = scratch(pkv), scratch(pkv, SIDE)
    more = scratch(pkv, SIDE, "small", True, need=2 * NEED)
    assert more is not side and scratch(pkv, SIDE) is more
    assert scratch(pkv) is main


@pytest.mark.parametrize("e4m3", [False, True])
def test_more_pairs_than_the_merge_counts(built, e4m3):
    """The tensor-core form numbers 32 pieces of every (sequence, KV head) pair in 32
    bits; calls of more pairs run on CUDA cores and need no workspace."""
    import ctypes
    size = built.lib.pkv_chunk_workspace_size_e4m3 if e4m3 else built.lib.pkv_chunk_workspace_size

    def on_tensor_cores(hkv, batch, tokens):
        d = built.CacheDesc(1000, 16, hkv, 128, 128)
        return size(ctypes.byref(d), tokens, batch, hkv, 64, 0) > 0
    most = ((1 << 31) - 1 - 256 * 64 - 256 * 8 * 8) // 32
    for hkv in (1, 8, 1023, 1024, 1025, 4096, 8191):
        batch = min(65535, most // hkv)
        assert on_tensor_cores(hkv, batch - 2048, batch - 2048)
        assert on_tensor_cores(hkv, batch, 5)
        if hkv >= 1025:
            assert not on_tensor_cores(hkv, batch + 2, batch + 2)


def test_withhold_control_is_for_the_tensor_core_form(built):
    """Refused, before anything is launched, wherever another kernel would run."""
    import ctypes
    p = ctypes.c_void_p(0x1000)

    def call(desc=(16, 16, 8, 128, 128), v=p, flags=0x100):
        d = built.CacheDesc(*desc)
        return built.lib.pkv_paged_chunk_attn(ctypes.byref(d), p, 4, 32, p, 2, p, v, p, 4, p, 1.0,
                                              0, 0, None, 0, p, p, flags, None)
    assert call() == -1
    built.lib.pkv_test_enable_withhold(1)
    try:
        assert call(flags=0x101) == -1 and call(flags=0x102) == -1 and call(flags=0x104) == -1
        assert call(desc=(16, 16, 8, 96, 96)) == -1 and call(v=None) == -1
        assert call() == -4                   # taken; it brings no workspace
    finally:
        built.lib.pkv_test_enable_withhold(0)
    assert call() == -1


@pytest.fixture
def calls(pkv, monkeypatch):
    """The arguments that reach the C calls, as C gets them (nothing runs)."""
    import ctypes
    seen = {}

    def stand_in(name):
        types = pkv.m._lib.SIGNATURES[name][1]

        def call(*args):
            seen[name] = [t(x).value if t in (ctypes.c_int32, ctypes.c_int64) else x
                          for t, x in zip(types, args)]
            return 0
        return call
    lib = SimpleNamespace(**{n: stand_in(n) for n in (
        "pkv_paged_chunk_attn", "pkv_paged_chunk_attn_e4m3", "pkv_rope_append",
        "pkv_rope_append_e4m3", "pkv_chunk_workspace_size", "pkv_chunk_workspace_size_e4m3")})
    monkeypatch.setattr(pkv.m, "lib", lib)
    return pkv.m, seen


NUMBERS = [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
           (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 16, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1),
           (-1, -1), (-2 ** 32 + 5, -1), (-2 ** 31 - 1, -1)]


@pytest.mark.parametrize("given,want", NUMBERS)
@pytest.mark.parametrize("e4m3", [False, True])
def test_numbers_past_32_bits(calls, given, want, e4m3):
    """A window or sinks past 2^31 see what 2^31 - 1 do, and a negative number or an
    offset past every head stays one that the call refuses: none wraps around."""
    m, seen = calls
    kind = torch.uint8 if e4m3 else torch.bfloat16
    pool = torch.zeros(4, 2, 16, 128, dtype=kind)
    scales = (torch.ones(2), torch.ones(2)) if e4m3 else ()
    q, cu, lens = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(2), torch.zeros(1)
    call = m.paged_chunk_attn_e4m3 if e4m3 else m.paged_chunk_attn
    call(q, cu, pool, pool, *scales, torch.zeros(1, 4), lens, 1.0, window=given, sink_tokens=given)
    args = seen["pkv_paged_chunk_attn_e4m3" if e4m3 else "pkv_paged_chunk_attn"]
    at = 14 if e4m3 else 12
    assert args[at:at + 2] == [want, want]
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    i64 = torch.zeros(3, dtype=torch.int64)
    if e4m3:
        m.rope_append_e4m3(pool, pool, q, k, k, i64, i64, torch.zeros(4), *scales,
                           rotary_offset=given)
    else:
        m.rope_append(pool, pool, q, k, k, i64, i64, torch.zeros(4), rotary_offset=given)
    args = seen["pkv_rope_append_e4m3" if e4m3 else "pkv_rope_append"]
    assert args[14 if e4m3 else 12] == want


@pytest.mark.parametrize("tokens", [1 << 29, 1 << 32, 1 << 59, 1 << 60, (1 << 60) + 4, 1 << 62])
def test_token_counts_whose_rows_pass_64_bits(built, tokens):
    """num_tokens * num_q_heads (16) wraps to a small number from 2^60 on."""
    import ctypes
    p = ctypes.c_void_p(0x1000)
    d = built.CacheDesc(16, 16, 8, 128, 128)
    rc = built.lib.pkv_paged_chunk_attn(ctypes.byref(d), p, tokens, 16, p, 2, p, p, p, 4, p, 1.0,
                                        0, 0, None, 0, p, p, 0, None)
    assert rc == -2
    assert built.lib.pkv_chunk_workspace_size(ctypes.byref(d), tokens, 2, 16, 4, 0) == 0


def test_a_workspace_the_gpu_cannot_write_is_refused(pkv, monkeypatch):
    """A workspace on the host, or one with gaps: as for every other buffer."""
    checked = []

    def need(t, name, dtype, dim=None):
        if name == "workspace":
            checked.append(name)
            if not t.is_contiguous():
                raise ValueError(name)
            raise TypeError(name)           # every tensor here is on the host
    monkeypatch.setattr(pkv.m, "_need", need)
    with pytest.raises(TypeError):
        scratch(pkv, None, "enough")
    with pytest.raises(TypeError):
        scratch(pkv, SIDE, "small", True)
    assert len(checked) == 2
    scratch(pkv)                            # none brought: nothing to check
    assert len(checked) == 2
