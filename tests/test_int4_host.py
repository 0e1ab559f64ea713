"""Host checks of the 4-bit cache's calls, the device-side tables' and the rotary
positions' of several axes, and the binding's own: nothing here reaches a GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests import _int4


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    return m


P, BAD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
DESC = (16, 16, 8, 128, 128)


def append(pkv, desc=DESC, k=P, kp=P, v=P, vp=P, kn=P, vn=P, slots=P, T=4):
    d = pkv.CacheDesc(*desc)
    return pkv.lib.pkv_kv_append_int4(ctypes.byref(d), k, kp, v, vp, kn, vn, slots, T, None)


def copy(pkv, desc=DESC, k=P, kp=P, v=P, vp=P, src=P, dst=P, n=4):
    d = pkv.CacheDesc(*desc)
    return pkv.lib.pkv_copy_blocks_int4(ctypes.byref(d), k, kp, v, vp, src, dst, n, None)


def decode(pkv, desc=DESC, q=P, batch=2, T=None, hq=32, k=P, kp=P, v=P, vp=P, tables=P, mb=4,
           lens=P, scale=1.0, S=1, ws=None, nbytes=0, out=P, lse=P, flags=0, partial=False):
    d = pkv.CacheDesc(*desc)
    head, pools = (ctypes.byref(d), q, batch), (hq, k, kp, v, vp, tables, mb, lens, scale, S)
    if partial:
        return pkv.lib.pkv_paged_decode_attn_partial_int4(*head, *pools, out, lse, flags, None)
    if T is not None:
        return pkv.lib.pkv_paged_decode_attn_multi_int4(*head, T, *pools, ws, nbytes, out, lse,
                                                        flags, None)
    return pkv.lib.pkv_paged_decode_attn_int4(*head, *pools, ws, nbytes, out, lse, flags, None)


BAD_DESCS = [((0, 16, 8, 128, 128), -1), ((16, 0, 8, 128, 128), -1), ((16, 257, 8, 128, 128), -1),
             ((16, 16, 0, 128, 128), -1), ((16, 16, 8, 0, 128), -1), ((16, 16, 8, 48, 128), -2),
             ((16, 16, 8, 128, 1056), -2), ((16, 16, 8, 128, 72), -2)]


@pytest.mark.parametrize("desc,status", BAD_DESCS)
def test_shapes(pkv, desc, status):
    assert append(pkv, desc) == copy(pkv, desc) == decode(pkv, desc) == status
    assert decode(pkv, desc, T=2) == decode(pkv, desc, partial=True) == status
    d = pkv.CacheDesc(*desc)
    assert pkv.lib.pkv_rope_append_int4(ctypes.byref(d), P, P, P, P, P, 32, P, P, P, 1, None, P, 4,
                                        P, 2, 0, 1.0, 0, P, None) == status
    assert pkv.lib.pkv_decode_workspace_size_int4(ctypes.byref(d), 2, 1, 32, 64, 3, 0) == 0


def test_append_and_copy_refusals(pkv):
    for name in ("k", "kp", "v", "vp", "kn", "vn", "slots"):
        assert append(pkv, **{name: None}) == -1, name
    for name in ("k", "kp", "v", "vp", "kn", "vn"):
        assert append(pkv, **{name: BAD}) == -3, name
    assert append(pkv, T=-1) == -1 and append(pkv, T=0, k=None) == 0
    assert append(pkv, T=1 << 60) == -2
    for name in ("k", "kp", "v", "vp", "src", "dst"):
        assert copy(pkv, **{name: None}) == -1, name
    for name in ("k", "kp", "v", "vp"):
        assert copy(pkv, **{name: BAD}) == -3, name
    assert copy(pkv, n=-1) == -1 and copy(pkv, n=0, k=None) == 0 and copy(pkv, n=65536) == -2


@pytest.mark.parametrize("form", [dict(), dict(T=2), dict(partial=True)])
def test_decode_refusals(pkv, form):
    for name in ("q", "k", "kp", "v", "vp", "tables", "lens", "out", "lse"):
        assert decode(pkv, **form, **{name: None}) == -1, name
    for name in ("q", "k", "kp", "v", "vp", "out"):
        assert decode(pkv, **form, **{name: BAD}) == -3, name
    for kw in (dict(batch=-1), dict(hq=0), dict(mb=-1), dict(S=-1), dict(S=257), dict(flags=4),
               dict(flags=0x100)):
        assert decode(pkv, **form, **kw) == -1, kw
    assert decode(pkv, **form, hq=12) == -2 and decode(pkv, **form, batch=65536) == -2
    assert decode(pkv, **form, hq=8 * 32768) == -2
    assert decode(pkv, **form, batch=0, q=None) == 0


def test_decode_workspace_and_tokens(pkv):
    need = pkv.lib.pkv_decode_workspace_size(2, 32, 128, 3)
    assert decode(pkv, S=3) == -4 and decode(pkv, S=3, ws=P, nbytes=need - 1) == -4
    assert decode(pkv, S=3, ws=BAD, nbytes=need) == -3
    need = pkv.lib.pkv_decode_workspace_size(2 * 5, 32, 128, 3)
    assert decode(pkv, T=5, S=3, ws=P, nbytes=need - 1) == -4
    assert decode(pkv, T=0) == -1 and decode(pkv, T=65) == -1
    assert decode(pkv, T=64, batch=1024) == -2
    assert decode(pkv, partial=True, S=0) == -1


def tables(pkv, trim=False, bs=16, nb=8, t=P, lens=P, change=P, batch=2, mb=4, free=P, state=P,
           rows=4, cu=P, pos=P, slots=P):
    if trim:
        return pkv.lib.pkv_trim_sequences(bs, nb, t, lens, change, batch, mb, free, state, None)
    return pkv.lib.pkv_extend_sequences(bs, nb, t, lens, change, batch, mb, free, state, rows, cu,
                                        pos, slots, None)


@pytest.mark.parametrize("trim", [False, True])
def test_tables_refusals(pkv, trim):
    for name in ("t", "lens", "change", "free", "state"):
        assert tables(pkv, trim, **{name: None}) == -1, name
    for kw in (dict(bs=0), dict(bs=257), dict(nb=0), dict(batch=-1), dict(mb=-1)):
        assert tables(pkv, trim, **kw) == -1, kw
    assert tables(pkv, trim, batch=8193) == -2
    assert tables(pkv, trim, batch=8192, mb=1 << 18) == -2
    if trim:
        assert tables(pkv, True, batch=0, t=None) == 0
    else:
        for name in ("cu", "pos", "slots"):
            assert tables(pkv, **{name: None}) == -1, name
        assert tables(pkv, rows=-1) == -1
        assert tables(pkv, pos=BAD) == -3 and tables(pkv, slots=BAD) == -3


def axes(pkv, e4m3=False, n=3, axis=P, **kw):
    d = pkv.CacheDesc(*kw.get("desc", DESC))
    rest = (P, n, axis, P, kw.get("T", 4), P, kw.get("rot", 128), 0, 1.0, kw.get("flags", 0),
            ctypes.c_void_p(0x2000), None)
    if e4m3:
        return pkv.lib.pkv_rope_append_axes_e4m3(ctypes.byref(d), P, P, P, 32, P, P,
                                                 kw.get("ks", P), P, *rest)
    return pkv.lib.pkv_rope_append_axes(ctypes.byref(d), P, P, P, 32, P, P, *rest)


@pytest.mark.parametrize("e4m3", [False, True])
def test_axes_refusals(pkv, e4m3):
    assert axes(pkv, e4m3, n=0) == axes(pkv, e4m3, n=9) == axes(pkv, e4m3, axis=None) == -1
    assert axes(pkv, e4m3, flags=4) == -1 and axes(pkv, e4m3, rot=130) == -2
    assert axes(pkv, e4m3, T=0) == 0
    if e4m3:
        assert axes(pkv, True, ks=None) == -1


def test_rope_int4_refusals(pkv):
    def call(k=P, kp=P, v=P, vp=P, n=1, axis=None, vn=P, q_out=ctypes.c_void_p(0x2000)):
        d = pkv.CacheDesc(*DESC)
        return pkv.lib.pkv_rope_append_int4(ctypes.byref(d), k, kp, v, vp, P, 32, P, vn, P, n,
                                            axis, P, 4, P, 128, 0, 1.0, 0, q_out, None)
    for name in ("k", "kp", "vp", "q_out"):
        assert call(**{name: None}) == -1, name
    assert call(v=None) == call(v=None, vn=None) == -1
    for name in ("k", "kp", "v", "vp"):
        assert call(**{name: BAD}) == -3, name
    assert call(n=2) == call(n=9, axis=P) == -1


@pytest.fixture
def cpu(pkv, monkeypatch):
    """The binding's checks with CPU tensors let through."""
    real = pkv._need

    def need(t, name, dtype, dim=None):
        class OnGpu:
            is_cuda, shape = True, t.shape
            dtype = t.dtype
            def is_contiguous(self): return t.is_contiguous()
            def dim(self): return t.dim()
        real(OnGpu(), name, dtype, dim)
    monkeypatch.setattr(pkv, "_need", need)
    monkeypatch.setattr(pkv, "_stream", lambda s=None: 0)
    return pkv


def test_the_binding_checks_its_tensors(cpu):
    c = _int4.make(1, [20, 3], 8, 2, 128, 128, 16)
    q, pools = c.q[:, 0].contiguous(), [c.k, c.k_params, c.v, c.v_params]

    def refused(kind, call, *args, **kw):
        with pytest.raises(kind):
            call(*args, **kw)

    def attn(q_=q, p=pools, t=c.tables, n=c.lens, **kw):
        return cpu.paged_decode_attn_int4(q_, *p, t, n, 0.1, **kw)
    refused(TypeError, attn, q.bfloat16())
    refused(ValueError, attn, q[:, :, :64].contiguous())
    refused(ValueError, attn, q[:1])
    refused(ValueError, attn, n=c.lens[:1])
    refused(ValueError, attn, q.transpose(0, 1))
    refused(TypeError, attn, p=[c.k.bfloat16(), *pools[1:]])
    refused(ValueError, attn, p=[c.k, c.k_params[:, :, :8].contiguous(), *pools[2:]])
    refused(ValueError, attn, p=[*pools[:2], c.v[:, :1].contiguous(), c.v_params[:, :1].contiguous()])
    refused(ValueError, attn, p=[*pools[:2], cpu.ValuesInKeys(64), c.v_params])
    refused(ValueError, attn, out=torch.empty(2, 8, 64))
    refused(ValueError, attn, lse=torch.empty(2, 4))
    refused(ValueError, attn, workspace=torch.empty(64, 64).t()[:32])
    refused(cpu.PkvError, attn, num_splits=257, workspace=torch.empty(1 << 22))
    refused(cpu.PkvError, attn, num_splits=2 ** 32 + 1, workspace=torch.empty(1 << 22))
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    refused(ValueError, cpu.kv_append_int4, *pools, x[:2], x, slots)
    refused(ValueError, cpu.kv_append_int4, *pools, x, x[..., :64].contiguous(), slots)
    refused(TypeError, cpu.kv_append_int4, *pools, x, x.float(), slots)
    refused(ValueError, cpu.copy_blocks_int4, *pools, c.lens, c.lens[:1])
    free, state = cpu.block_pool(9, device="cpu", order=[2, 0, 1, 3, 4, 5, 6, 7, 8])
    assert free.tolist() == [8, 7, 6, 5, 4, 3, 1, 0, 2] and state.tolist() == [9, 0, 0, 0]
    refused(ValueError, cpu.block_pool, 3, "cpu", [0, 0, 1])
    ext = (c.tables, c.lens, c.lens, free, state, 16)
    refused(ValueError, cpu.extend_sequences, *ext, -1)
    refused(ValueError, cpu.extend_sequences, *ext, 2 ** 31)
    refused(ValueError, cpu.extend_sequences, c.tables, c.lens, c.lens[:1], *ext[3:], 4)
    refused(ValueError, cpu.extend_sequences, *ext, 4, cu_q_lens=c.lens)
    refused(ValueError, cpu.extend_sequences, *ext, 4, slots=slots)
    refused(ValueError, cpu.extend_sequences, *ext[:4], state[:2], 16, 4)
    refused(cpu.PkvError, cpu.extend_sequences, *ext[:5], 2 ** 32 + 16, 4)
    refused(ValueError, cpu.trim_sequences, c.tables[:1], *ext[1:])
    refused(TypeError, cpu.trim_sequences, c.tables, c.lens.long(), *ext[2:])
    inv = torch.zeros(64, dtype=torch.float64)
    axis = torch.zeros(64, dtype=torch.int32)
    bf = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    rope = (x, x, x)
    refused(ValueError, cpu.rope_append, bf, bf, *rope, slots, slots, inv, pair_axis=axis)
    refused(ValueError, cpu.rope_append, bf, bf, *rope, slots[None], slots, inv)
    refused(ValueError, cpu.rope_append, bf, bf, *rope, slots[None], slots, inv,
            pair_axis=axis[:3])
    refused(ValueError, cpu.rope_append, bf, bf, *rope, slots[None].repeat(9, 1), slots, inv,
            pair_axis=axis)
    refused(ValueError, cpu.rope_append_int4, *pools, *rope, slots[None, :2], slots, inv,
            pair_axis=axis)


def test_the_rows_format():
    """The plain quantiser itself: half a step, whole rows, odd rows."""
    x = torch.randn(500, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes, params = _int4.quantise(x)
    back = _int4.values(codes, params)
    s = params[:, :1].double()
    top = params[:, 1:].double() + 15 * s
    err = (back - x.double()).abs()
    assert torch.all(err <= s / 2 * (1 + 2.0 ** -18) + (x.double() - top).clamp_min(0))
    for v, p in ((torch.full((1, 32), 3.0), (0.0, 3.0)), (torch.zeros(1, 32), (0.0, 0.0))):
        codes, params = _int4.quantise(v)
        assert torch.all(codes == 0) and params[0].tolist() == list(p)
    v = torch.randn(1, 32)
    v[0, 3] = float("inf")
    codes, params = _int4.quantise(v)
    assert torch.all(codes == 0) and params.isnan().all()
