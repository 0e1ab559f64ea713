"""Rotary positions fused with the append (pkv_rope_append and its E4M3 form)
against the definition in 64 bits, and a run of append, prompt attention and
decode steps as they are used together."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    m.device_status(reset=True)
    return m


def turned(x, pos, inv_freq, off, interleaved, amplitude):
    """x [T, H, D] float64 rotated, and |x1| + |x2| at every element."""
    rot = 2 * inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y, size = x.clone(), torch.zeros_like(x)
    part = x[..., off:off + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        i1, i2 = slice(off, off + rot, 2), slice(off + 1, off + rot, 2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        i1, i2 = slice(off, off + rot // 2), slice(off + rot // 2, off + rot)
    y[..., i1], y[..., i2] = amplitude * (a * c - b * s), amplitude * (b * c + a * s)
    size[..., i1] = size[..., i2] = amplitude * (a.abs() + b.abs())
    return y, size


def close(got, ref, size, kind, scale=None):
    """fp32: the angle's fraction of a turn is rounded to binary32 (pi 2^-24)
    and cos and sin are within 2 ulp (2^-23), two products and a sum: under
    8e-7 of |x1| + |x2|.  bf16 adds half a step, 2^-8 of the value; E4M3 the
    quotient's 2^-4, or half the smallest step, 2^-10."""
    got = got.cpu().double()
    tol = 8e-7 * size
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    elif kind == "e4m3":
        got, ref = got, (ref / scale).clamp(-448, 448)
        tol = tol / scale + torch.maximum(2.0 ** -4 * (ref.abs() + tol / scale),
                                          torch.tensor(2.0 ** -10, dtype=torch.float64))
    err = (got - ref).abs()
    assert torch.all(err <= tol), float((err - tol).max())


def make(seed, T, hq, hkv, dk, dv, bs, e4m3=False, far=200000):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    nb = -(-T // bs) + 2
    t = dict(q=torch.randn(T, hq, dk, generator=g).to(bf),
             k=torch.randn(T, hkv, dk, generator=g).to(bf),
             v=None if dv is None else torch.randn(T, hkv, dv, generator=g).to(bf),
             pos=torch.randint(0, far, (T,), generator=g),
             slots=torch.randperm(nb * bs, generator=g)[:T].clone())
    pools = []
    for d in (dk, dv):
        if d is None:
            pools.append(None)
        elif e4m3:
            pools.append(torch.randint(0, 120, (nb, hkv, bs, d), generator=g).to(torch.uint8))
        else:
            pools.append(torch.randn(nb, hkv, bs, d, generator=g).to(bf))
    t["kp"], t["vp"] = pools
    if e4m3:
        t["ks"] = (3 + torch.rand(hkv, generator=g)) / 448
        t["vs"] = (3 + torch.rand(hkv, generator=g)) / 448
    return t


def call(pkv, t, inv, latent_dv=None, dev="cuda", **kw):
    d = {n: (None if x is None else x.to(dev)) for n, x in t.items()}
    vp = pkv.ValuesInKeys(latent_dv) if t["vp"] is None else d["vp"]
    if "ks" in t:
        q = pkv.rope_append_e4m3(d["kp"], vp, d["q"], d["k"], d["v"], d["pos"], d["slots"],
                                 inv.to(dev), d["ks"], d["vs"], **kw)
    else:
        q = pkv.rope_append(d["kp"], vp, d["q"], d["k"], d["v"], d["pos"], d["slots"],
                            inv.to(dev), **kw)
    torch.cuda.synchronize()
    return q, d["kp"], d["vp"]


def rows(pool, slots, bs):
    s = slots.to(pool.device)
    return pool[s // bs, :, s % bs]


def check(t, inv, got, off=0, interleaved=False, amplitude=1.0, fp32=False, live=None):
    q, kp, vp = got
    live = torch.arange(t["pos"].numel()) if live is None else live
    ref, size = turned(t["q"].double(), t["pos"], inv, off, interleaved, amplitude)
    if fp32:
        assert q.dtype == torch.float32
    close(q.cpu()[live], ref[live], size[live], "fp32" if fp32 else "bf16")
    bs = t["kp"].shape[2]
    ref, size = turned(t["k"].double(), t["pos"], inv, off, interleaved, amplitude)
    slots = t["slots"][live]
    if "ks" in t:
        e4 = torch.float8_e4m3fn
        close(rows(kp.cpu().view(e4).double(), slots, bs), ref[live], size[live], "e4m3",
              t["ks"].double()[None, :, None])
        close(rows(vp.cpu().view(e4).double(), slots, bs), t["v"].double()[live],
              torch.zeros(()), "e4m3", t["vs"].double()[None, :, None])
    else:
        close(rows(kp, slots, bs), ref[live], size[live], "bf16")
        if vp is not None:
            assert torch.equal(rows(vp, slots, bs).cpu(), t["v"][live])
    # every other row of the pools is as it was
    for new, old in ((kp, t["kp"]), (vp, t["vp"])):
        if new is None:
            continue
        new, old = new.cpu().transpose(1, 2).flatten(0, 1), old.transpose(1, 2).flatten(0, 1)
        rest = torch.ones(old.shape[0], dtype=torch.bool)
        rest[slots] = False
        assert torch.equal(new[rest], old[rest])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("shape", [(32, 8, 128, 128, 16), (4, 2, 64, 64, 4), (5, 1, 128, 64, 8),
                                   (3, 3, 72, 40, 5)])
def test_full_and_partial(pkv, shape, T, interleaved):
    hq, hkv, dk, dv, bs = shape
    for rot, off in ((dk, 0), (dk // 2, 0), (dk // 2, dk // 2), (2, 6), (24, 8), (dk - 2, 1)):
        t = make(T + rot, T, hq, hkv, dk, dv, bs)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        for fp32 in (False, True):
            got = call(pkv, t, inv, rotary_offset=off, interleaved=interleaved, amplitude=1.25,
                       q_dtype=torch.float32 if fp32 else torch.bfloat16)
            check(t, inv, got, off, interleaved, 1.25, fp32)
    assert pkv.device_status(reset=True) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,off", [(128, 0), (64, 64), (6, 3)])
def test_e4m3(pkv, interleaved, rot, off):
    t = make(3, 45, 16, 4, 128, 128, 16, e4m3=True)
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / 8
    check(t, inv, call(pkv, t, inv, rotary_offset=off, interleaved=interleaved), off, interleaved)


def test_latent_rows(pkv):
    t = make(4, 33, 128, 1, 576, None, 64)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    check(t, inv, call(pkv, t, inv, latent_dv=512, rotary_offset=512, interleaved=True), 512, True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(pkv, interleaved):
    t = make(5, 50, 8, 2, 128, 128, 16)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    want = call(pkv, t, inv, rotary_offset=32, interleaved=interleaved)[0]
    dev = "cuda"
    q = t["q"].to(dev)
    got = pkv.rope_append(t["kp"].to(dev), t["vp"].to(dev), q, t["k"].to(dev), t["v"].to(dev),
                          t["pos"].to(dev), t["slots"].to(dev), inv.to(dev), rotary_offset=32,
                          interleaved=interleaved, q_out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q, want)


def test_far_positions(pkv):
    """Positions past 2^31 and 2^40 keep their angle."""
    t = make(6, 64, 4, 1, 128, 128, 16)
    t["pos"] = torch.arange(64) * 977 + 2 ** 31 - 30000
    inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    check(t, inv, call(pkv, t, inv, q_dtype=torch.float32), fp32=True)
    # whole quarter turns: exact whatever the position
    t["pos"] = torch.arange(64) * 12345 + 2 ** 40
    quarter = torch.full((64,), math.pi / 2, dtype=torch.float64)
    q = call(pkv, t, quarter, q_dtype=torch.float32)[0].cpu().double()
    k = (t["pos"] % 4)[:, None, None]
    x = t["q"].double()
    a, b = x[..., :64], x[..., 64:]
    ref = torch.cat([torch.where(k == 0, a, torch.where(k == 1, -b, torch.where(k == 2, -a, b))),
                     torch.where(k == 0, b, torch.where(k == 1, a, torch.where(k == 2, -b, -a)))],
                    -1)
    # pi / 2 is a binary64: off by 2^-54 relative, 2^40 quarter turns by 1e-4 of a radian
    assert float((q - ref).abs().max()) < 2e-3


def test_padding_and_slots(pkv):
    t = make(7, 20, 8, 2, 128, 128, 16)
    inv = 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)
    t["pos"][3] = t["pos"][19] = -1
    t["slots"][5] = -1
    dev = "cuda"
    q = torch.full(t["q"].shape, 7.0, dtype=torch.bfloat16, device=dev)
    got = call(pkv, t, inv, q_out=q)
    assert pkv.device_status(reset=True) == 0
    assert torch.all(q[3] == 7) and torch.all(q[19] == 7)
    live = torch.tensor([i for i in range(20) if i not in (3, 5, 19)])
    check(t, inv, got, live=live)
    ref, size = turned(t["q"].double(), t["pos"], inv, 0, False, 1.0)
    close(q.cpu()[5:6], ref[5:6], size[5:6], "bf16")
    t["slots"][6] = t["kp"].shape[0] * 16
    t["slots"][7] = 2 ** 62
    got = call(pkv, t, inv)
    assert pkv.device_status(reset=True) == pkv.DEV_SLOT
    check(t, inv, got, live=torch.tensor([i for i in live.tolist() if i not in (6, 7)]))


def test_graph_replay(pkv):
    dev = "cuda"
    t = make(8, 9, 8, 2, 128, 128, 16)
    u = make(9, 9, 8, 2, 128, 128, 16)
    inv = pkv.rope_frequencies(128)
    d = {n: x.to(dev) for n, x in t.items()}
    q = torch.empty_like(d["q"])
    step = lambda: pkv.rope_append(d["kp"], d["vp"], d["q"], d["k"], d["v"], d["pos"], d["slots"],
                                   inv, q_out=q)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in d:
        d[n].copy_(u[n])
    graph.replay()
    torch.cuda.synchronize()
    check(u, inv.cpu(), (q, d["kp"], d["vp"]))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_served_sequence(pkv, e4m3):
    """Two prompts in chunks, then single tokens, through rope_append and
    chunk attention under a window with sinks: each token's output equals
    attention over all rotated keys computed at once in 64 bits."""
    from tests import _chunk
    dev, bf = "cuda", torch.bfloat16
    hq, hkv, D, bs, W, S = 8, 2, 128, 16, 48, 3
    g = torch.Generator().manual_seed(31)
    total = [150, 77]
    q = [torch.randn(n, hq, D, generator=g).to(bf) for n in total]
    k = [torch.randn(n, hkv, D, generator=g).to(bf) for n in total]
    v = [torch.randn(n, hkv, D, generator=g).to(bf) for n in total]
    nb = 20
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.stack([perm[:10], perm[10:]]).to(dev)
    kp = torch.zeros(nb, hkv, bs, D, dtype=torch.uint8 if e4m3 else bf, device=dev)
    vp = torch.zeros_like(kp)
    ks, vs = (torch.full((hkv,), 5 / 448, device=dev) for _ in range(2))
    inv = pkv.rope_frequencies(D, theta=10000.0, factor=4.0, original_len=64, device=dev)
    done, outs, qs = [0, 0], [[], []], [[], []]
    for news in ([100, 0], [37, 60], [1, 16], [1, 1], [11, 0]):
        cat = lambda x: torch.cat([x[b][done[b]:done[b] + n] for b, n in enumerate(news)]).to(dev)
        pos = torch.cat([torch.arange(done[b], done[b] + n) for b, n in enumerate(news)]).to(dev)
        seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(news)]).to(dev)
        slots = pkv.slot_mapping(kp, vp, tables, seq, pos)
        new = (cat(q), cat(k), cat(v), pos, slots, inv)
        if e4m3:
            qr = pkv.rope_append_e4m3(kp, vp, *new, ks, vs)
        else:
            qr = pkv.rope_append(kp, vp, *new)
        done = [d + n for d, n in zip(done, news)]
        cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=dev)
        lens = torch.tensor(done, dtype=torch.int32, device=dev)
        rest = (tables, lens, D ** -0.5)
        if e4m3:
            out, _ = pkv.paged_chunk_attn_e4m3(qr, cu, kp, vp, ks, vs, *rest, window=W,
                                               sink_tokens=S)
        else:
            out, _ = pkv.paged_chunk_attn(qr, cu, kp, vp, *rest, window=W, sink_tokens=S)
        for b, part in enumerate(out.split(news)):
            outs[b].append(part)
        for b, part in enumerate(qr.split(news)):
            qs[b].append(part)
    torch.cuda.synchronize()
    assert done == total and pkv.device_status(reset=True) == 0
    # the rotated queries and keys are the definition's, the outputs attention over the cache
    for b in range(2):
        ref, size = turned(q[b].double(), torch.arange(total[b]), inv.cpu(), 0, False, 1.0)
        close(torch.cat(qs[b]), ref, size, "bf16")
        case = _chunk.ChunkCase(torch.cat(qs[b]).cpu(), torch.tensor([0, total[b]]).int(),
                                kp.cpu(), vp.cpu(), D, tables[b:b + 1].cpu(),
                                torch.tensor([total[b]]).int(), D ** -0.5, W, S,
                                ks.cpu() if e4m3 else None, vs.cpu() if e4m3 else None)
        want = _chunk.reference(case)
        _chunk.check(case, torch.cat(outs[b]), want[1])


# enough tokens that every form works through several tokens and parts a thread
@pytest.mark.parametrize("T,shape,rot,off,interleaved", [
    (6000, (8, 2, 128, 128, 16), 128, 0, False), (5003, (8, 2, 64, 64, 16), 32, 0, True),
    (5001, (4, 2, 256, 256, 16), 64, 64, False), (9000, (5, 1, 128, 64, 8), 64, 0, False),
    (20000, (3, 1, 64, 128, 8), 16, 8, True), (1300, (64, 2, 128, 128, 16), 128, 0, True),
    (5000, (2, 1, 72, 40, 5), 24, 3, False), (5500, (2, 2, 512, 512, 16), 128, 128, True)])
def test_many_tokens(pkv, T, shape, rot, off, interleaved):
    hq, hkv, dk, dv, bs = shape
    t = make(T, T, hq, hkv, dk, dv, bs)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    for fp32 in (False, True):
        got = call(pkv, t, inv, rotary_offset=off, interleaved=interleaved,
                   q_dtype=torch.float32 if fp32 else torch.bfloat16)
        check(t, inv, got, off, interleaved, fp32=fp32)


@pytest.mark.parametrize("T,shape,rot,off", [(6000, (4, 2, 128, 128, 16), 128, 0),
                                             (7000, (4, 2, 128, 64, 16), 64, 64),
                                             (5100, (3, 1, 72, 40, 16), 8, 0)])
def test_many_tokens_e4m3(pkv, T, shape, rot, off):
    hq, hkv, dk, dv, bs = shape
    t = make(T, T, hq, hkv, dk, dv, bs, e4m3=True)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    check(t, inv, call(pkv, t, inv, rotary_offset=off), off)


@pytest.mark.parametrize("T,interleaved", [(700, True), (2500, False)])
def test_many_latent_rows(pkv, T, interleaved):
    t = make(T, T, 32, 1, 576, None, 64)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    check(t, inv, call(pkv, t, inv, latent_dv=512, rotary_offset=512, interleaved=interleaved),
          512, interleaved)


def test_a_stream_of_ones_own(pkv):
    t = make(9, 40, 8, 2, 128, 128, 16)
    inv = pkv.rope_frequencies(128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(t, inv.cpu(), call(pkv, t, inv, stream=s))
