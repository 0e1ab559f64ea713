"""Rotary positions of several axes, and rotary positions into a 4-bit cache, against
their definitions in 64 bits; and a drafting server's steps as they follow one another:
tables extended on the device, rotary append, attention, the refused tokens trimmed."""
from __future__ import annotations

import math
import random

import pytest
import torch

from tests import _int4
from tests.test_gpu_rope import close, make, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    m.device_status(reset=True)
    return m


def turned(x, pos, axis, inv, off, interleaved, amplitude):
    """x [T, H, D] rotated, pair i by positions[axis[i]], and |x1| + |x2| everywhere."""
    x = x.double()
    rot = 2 * inv.numel()
    angle = torch.stack([pos[a].double() * f for a, f in zip(axis.tolist(), inv)], 1)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    first = [off + (2 * i if interleaved else i) for i in range(rot // 2)]
    second = [e + (1 if interleaved else rot // 2) for e in first]
    a, b = x[..., first], x[..., second]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = amplitude * (a * c - b * s), amplitude * (b * c + a * s)
    size[..., first] = size[..., second] = amplitude * (a.abs() + b.abs())
    return y, size


def inputs(seed, T, axes, rot, far=5000):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, far, (axes, T), generator=g)
    if axes > 1:
        pos[1:] -= far // 3                       # axes may be centred
    axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.int32)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return pos, axis, inv


def on_gpu(t):
    return {n: None if x is None else x.cuda() for n, x in t.items()}


# hq, hkv, dk, dv, bs, rot, off: one for each kernel form
FORMS = [(32, 8, 128, 128, 16, 128, 0), (28, 4, 64, 64, 8, 32, 16), (5, 1, 160, 64, 8, 64, 16),
         (3, 3, 72, 40, 5, 22, 7), (2, 2, 96, 96, 16, 64, 8)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,axes", [(1, 3), (50, 2), (301, 3), (20, 8), (9, 1)])
@pytest.mark.parametrize("form", FORMS)
def test_axes(pkv, form, T, axes, interleaved):
    hq, hkv, dk, dv, bs, rot, off = form
    for e4m3 in (False, True):
        t = make(T + rot, T, hq, hkv, dk, dv, bs, e4m3=e4m3)
        pos, axis, inv = inputs(T, T, axes, rot)
        d = on_gpu(t)
        scales = (d["ks"], d["vs"]) if e4m3 else ()
        q = (pkv.rope_append_e4m3 if e4m3 else pkv.rope_append)(
            d["kp"], d["vp"], d["q"], d["k"], d["v"], pos.cuda(), d["slots"], inv.cuda(), *scales,
            rotary_offset=off, interleaved=interleaved, amplitude=1.25, q_dtype=torch.float32,
            pair_axis=axis.cuda())
        how = (pos, axis, inv, off, interleaved, 1.25)
        close(q, *turned(t["q"], *how), "fp32")
        got = rows(d["kp"].cpu().view(torch.float8_e4m3fn).double() if e4m3 else d["kp"],
                   t["slots"], bs)
        close(got, *turned(t["k"], *how), "e4m3" if e4m3 else "bf16",
              t["ks"].double()[None, :, None] if e4m3 else None)
        if not e4m3:
            assert torch.equal(rows(d["vp"], t["slots"], bs).cpu(), t["v"])
    assert pkv.device_status() == 0


def test_one_axis_is_the_plain_call(pkv):
    """Every pair on one axis: the plain call's bits, whichever axis that is."""
    t = make(3, 77, 16, 4, 128, 128, 16)
    pos, _, inv = inputs(3, 77, 3, 128)
    pos = pos.abs()
    for axis in range(3):
        d, e = on_gpu(t), on_gpu(t)
        # (axis 0 tells padding: none here)
        pair_axis = torch.full((64,), axis, dtype=torch.int32, device="cuda")
        a = pkv.rope_append(d["kp"], d["vp"], d["q"], d["k"], d["v"], pos.cuda(), d["slots"],
                            inv.cuda(), pair_axis=pair_axis)
        b = pkv.rope_append(e["kp"], e["vp"], e["q"], e["k"], e["v"], pos[axis].cuda(), e["slots"],
                            inv.cuda())
        assert torch.equal(a, b) and torch.equal(d["kp"], e["kp"])


@pytest.mark.parametrize("form", FORMS)
def test_padding_and_bad_axes(pkv, form):
    hq, hkv, dk, dv, bs, rot, off = form
    t = make(5, 12, hq, hkv, dk, dv, bs)
    pos, axis, inv = inputs(5, 12, 3, rot)
    pos[0, 4] = -1
    d = on_gpu(t)
    axis[1] = 3
    out = torch.full_like(d["q"], 7.0)
    pkv.rope_append(d["kp"], d["vp"], d["q"], d["k"], d["v"], pos.cuda(), d["slots"], inv.cuda(),
                    rotary_offset=off, q_out=out, pair_axis=axis.cuda())
    assert pkv.device_status() == pkv.DEV_AXIS
    axis[1] = 0
    live = [i for i in range(12) if i != 4]
    want, size = turned(t["q"], pos, axis, inv, off, False, 1.0)
    close(out[live], want[live], size[live], "bf16")
    assert torch.all(out[4] == 7)
    s = int(t["slots"][4])
    assert torch.equal(d["kp"][s // bs, :, s % bs].cpu(), t["kp"][s // bs, :, s % bs])


def check_int4(x, size, pool, params):
    """The stored rows [T, H, D] against what should be in them: x, of which the kernel's own
    is off by e = 8e-7 of `size` (the angle, cosine and sine, two products and a sum)."""
    e = 8e-7 * size
    params = params.double()
    s, o = params[..., :1], params[..., 1:]
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    slack = e.amax(-1, keepdim=True) + 2.0 ** -8 * low.abs()
    assert torch.all((o - low).abs() <= slack)
    spread = (high - o).clamp_min(0)
    # a rounding of the difference, of the product and of 1/15, and half a step of bf16
    assert torch.all((s - spread / 15).abs() <= (2.0 ** -8 + 2.0 ** -22) * (spread / 15) +
                     e.amax(-1, keepdim=True))
    back = torch.stack((pool & 15, pool >> 4), -1).flatten(-2).double() * s + o
    # half a step, and what lies past the row's ends
    outside = (x - (o + 15 * s)).clamp_min(0) + (o - x).clamp_min(0)
    assert torch.all((back - x).abs() <= 0.5 * s * (1 + 2.0 ** -18) + 2 * e + outside +
                     2.0 ** -22 * (x - o).abs())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,axes", [(1, 1), (45, 3), (300, 1)])
@pytest.mark.parametrize("form", [(32, 8, 128, 128, 16, 128, 0), (28, 4, 64, 64, 8, 32, 16),
                                  (4, 2, 256, 256, 4, 64, 64), (3, 1, 512, 512, 2, 128, 0),
                                  (5, 1, 160, 64, 8, 64, 16), (2, 2, 96, 96, 16, 90, 3),
                                  (6, 3, 32, 128, 5, 2, 30), (3, 1, 1024, 32, 4, 600, 200)])
def test_int4(pkv, form, T, axes, interleaved):
    hq, hkv, dk, dv, bs, rot, off = form
    t = make(T + rot, T, hq, hkv, dk, dv, bs)
    pos, axis, inv = inputs(T, T, axes, rot)
    if T > 2:
        pos[0, 1], t["slots"][2] = -1, -1
    nb = t["kp"].shape[0]
    g = torch.Generator().manual_seed(1)
    pools = [torch.randint(0, 256, (nb, hkv, bs, dk // 2), generator=g).to(torch.uint8),
             torch.ones(nb, hkv, bs, 2, dtype=torch.bfloat16),
             torch.randint(0, 256, (nb, hkv, bs, dv // 2), generator=g).to(torch.uint8),
             torch.ones(nb, hkv, bs, 2, dtype=torch.bfloat16)]
    for q_dtype in (torch.float32, torch.bfloat16):
        d, got = on_gpu(t), [p.cuda() for p in pools]
        q = pkv.rope_append_int4(
            *got, d["q"], d["k"], d["v"], pos.cuda() if axes > 1 else pos[0].cuda(), d["slots"],
            inv.cuda(), rotary_offset=off, interleaved=interleaved, amplitude=1.25,
            q_dtype=q_dtype, pair_axis=axis.cuda() if axes > 1 else None)
        assert pkv.device_status() == 0
        live = torch.tensor([i for i in range(T) if T <= 2 or i != 1])
        kept = torch.tensor([i for i in range(T) if T <= 2 or i not in (1, 2)])
        how = (pos, axis, inv, off, interleaved, 1.25)
        want, size = turned(t["q"], *how)
        close(q.cpu()[live], want[live], size[live],
              "fp32" if q_dtype == torch.float32 else "bf16")
        k, ksize = turned(t["k"], *how)
        slots = t["slots"][kept]
        back = [rows(p.cpu(), slots, bs) for p in got]
        check_int4(k[kept], ksize[kept], back[0], back[1])
        # values are not turned: the append's codes and parameters
        codes, params = _int4.quantise(t["v"][kept])
        assert torch.equal(back[2], codes) and torch.equal(back[3], params)
        rest = torch.ones(nb * bs, dtype=torch.bool)
        rest[slots] = False
        for new, old in zip(got, pools):
            new, old = new.cpu().transpose(1, 2).flatten(0, 1), old.transpose(1, 2).flatten(0, 1)
            assert torch.equal(new[rest], old[rest])


def test_int4_in_place(pkv):
    for hq, hkv, d, bs, rot, off in ((8, 2, 128, 16, 64, 32), (4, 2, 96, 16, 50, 7)):
        t = make(5, 50, hq, hkv, d, d, bs)
        t["q"][3, 1, 0] = float("nan")
        pos, axis, inv = inputs(5, 50, 3, rot)
        nb = t["kp"].shape[0]
        g = on_gpu(t)

        def call(q_out):
            pools = [torch.zeros(nb, hkv, bs, n, dtype=dt, device="cuda")
                     for _ in range(2) for n, dt in ((d // 2, torch.uint8), (2, torch.bfloat16))]
            return pkv.rope_append_int4(*pools, g["q"], g["k"], g["v"], pos.cuda(), g["slots"],
                                        inv.cuda(), rotary_offset=off, q_out=q_out,
                                        pair_axis=axis.cuda())
        want = call(None)
        assert torch.equal(want.view(torch.int16)[..., :off].cpu(),
                           t["q"].view(torch.int16)[..., :off])
        got = call(g["q"])
        assert got is g["q"] and torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("d,hq,hkv,bs", [(128, 32, 8, 16), (64, 14, 2, 32), (96, 4, 2, 8)])
def test_a_drafting_server(pkv, d, hq, hkv, bs):
    """Prompts, then steps of T drafted tokens of which some are refused: tables, positions
    and slots from the device, rotary positions of three axes, a 4-bit cache."""
    rng = random.Random(d)
    g = torch.Generator().manual_seed(d)
    B, T, axes = 5, 4, 3
    nb, width = 200, 40
    free, state = pkv.block_pool(nb, order=rng.sample(range(nb), nb))
    tables = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    pools = [torch.full((nb, hkv, bs, n), 255 if n > 2 else math.nan, dtype=dt, device="cuda")
             for _ in range(2) for n, dt in ((d // 2, torch.uint8), (2, torch.bfloat16))]
    _, axis, inv = inputs(1, 1, axes, d)
    kept = [[] for _ in range(B)]                 # each sequence's (k, v) rows in 64 bits

    def step(new):
        n = sum(new)
        rows_ = n + 3
        cu, positions, slots = pkv.extend_sequences(
            tables, lens, torch.tensor(new, dtype=torch.int32, device="cuda"), free, state, bs,
            rows_)
        x = {name: torch.randn(rows_, h, d, generator=g).to(torch.bfloat16)
             for name, h in (("q", hq), ("k", hkv), ("v", hkv))}
        # time, then two more axes that a program derives from it
        pos = torch.stack((positions, positions // 7, positions % 7))
        q = pkv.rope_append_int4(*pools, x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), pos, slots,
                                 inv.cuda(), q_dtype=torch.float32, pair_axis=axis.cuda())
        assert pkv.device_status() == 0
        at = 0
        for b, m in enumerate(new):
            first = len(kept[b])
            assert positions[at:at + m].tolist() == list(range(first, first + m))
            kept[b] += [None] * m
            at += m
        assert int(cu[-1]) == n and slots[n:].tolist() == [-1] * 3
        return q[:n], pos[:, :n].cpu(), x

    def attend(q, T_):
        c = _int4.Case(q.view(B, T_, hq, d).cpu(), *(p.cpu() for p in pools), tables.cpu(),
                       lens.cpu(), d ** -0.5)
        out, lse = pkv.paged_decode_attn_multi_int4(q.view(B, T_, hq, d), *pools, tables, lens,
                                                    d ** -0.5)
        assert pkv.device_status() == 0
        _int4.close(out, lse, _int4.attend(c))

    prompts = [rng.randint(1, 60) for _ in range(B)]
    step(prompts)
    for turn in range(4):
        q, pos, x = step([T] * B)
        # the rotated queries are what the positions say
        want, size = turned(x["q"][:B * T], pos, axis, inv, 0, False, 1.0)
        close(q, want, size, "fp32")
        attend(q, T)
        keep = [len(r) - rng.randint(0, T) for r in kept]
        if turn == 2:
            keep[1] = 0                           # done: all its blocks go back
        pkv.trim_sequences(tables, lens, torch.tensor(keep, dtype=torch.int32, device="cuda"),
                           free, state, bs)
        kept = [r[:n] for r, n in zip(kept, keep)]
        assert lens.tolist() == keep
        held = [tables[b, i].item() for b, n in enumerate(keep) for i in range(-(-n // bs))]
        count = int(state[0])
        assert sorted(held + free[:count].tolist()) == list(range(nb))
