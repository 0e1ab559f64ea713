"""Decode over a 4-bit cache as a server runs it: captured once and replayed with other
lengths, on streams of their own, with the library's plan and with given splits; two calls at
once, a padded batch, the appends captured with the attention."""
from __future__ import annotations

import pytest
import torch

from tests import _int4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    m.device_status(reset=True)
    return m


def call_of(pkv, c):
    """-> the call, its q and its other tensors."""
    multi = c.q.shape[1] > 1
    call = pkv.paged_decode_attn_multi_int4 if multi else pkv.paged_decode_attn_int4
    return call, (c.q if multi else c.q[:, 0]).contiguous().cuda(), [*c.pools(), c.tables.cuda()]


def with_lens(c, lens):
    return _int4.Case(c.q, c.k, c.k_params, c.v, c.v_params, c.tables,
                      torch.tensor(lens, dtype=torch.int32), c.scale)


@pytest.mark.parametrize("num_splits", [0, 1, 4])
@pytest.mark.parametrize("d", [128, 64, 96])
def test_replays_with_other_lengths(pkv, d, num_splits):
    """Two graphs, each with a workspace of its own, replayed at once, their lengths rewritten
    between the replays; and the same by direct calls on both streams."""
    cases = [_int4.make(61, [2600, 40, 0, 700], 16, 4, d, d, 16, 1, width=170),
             _int4.make(62, [900, 1700, 90], 8, 2, d, d, 16, 4, width=110)]
    turns = [([2600, 40, 0, 700], [900, 1700, 90]), ([0, 39, 0, 1], [4, 1699, 5]),
             ([129, 12, 0, 700], [899, 128, 89]), ([2600, 40, 0, 700], [900, 1700, 90])]
    made = []
    for c in cases:
        call, q, rest = call_of(pkv, c)
        lens, s = c.lens.cuda(), torch.cuda.Stream()
        B, T, Hq = c.q.shape[:3]
        need = pkv.decode_workspace_size_int4(*rest[:4], B, Hq, c.tables.shape[1], T, num_splits)
        # the plan's (heads of 64 and 128), or chunks' partials
        assert (need > 0) == (num_splits != 1)
        call(q, *rest, lens, c.scale, num_splits=num_splits)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call(q, *rest, lens, c.scale, num_splits=num_splits)
        made.append((c, call, q, rest, lens, s, graph, got))
    for at, turn in enumerate(turns):
        direct = []
        for (c, call, q, rest, lens, s, graph, got), now in zip(made, turn):
            s.wait_stream(torch.cuda.current_stream())
            new = torch.tensor(now, dtype=torch.int32).pin_memory()
            with torch.cuda.stream(s):
                lens.copy_(new, non_blocking=True)
                graph.replay()
            direct.append(call(q, *rest, lens, c.scale, num_splits=num_splits, stream=s))
        torch.cuda.synchronize()
        for (c, *_, got), now, (out, lse) in zip(made, turn, direct):
            _int4.close(*got, _int4.attend(with_lens(c, now)))
            assert torch.equal(got[0], out) and torch.equal(got[1], lse), at
            got[0].fill_(float("nan"))
        torch.cuda.synchronize()
    assert pkv.device_status() == 0


def test_many_calls_at_once(pkv):
    """Planned calls of other shapes on four streams, many in flight, each repeated exactly."""
    shapes = [([3000, 17, 900], 32, 8, 128, 1), ([1200] * 9, 64, 8, 128, 1),
              ([5000], 8, 1, 64, 3), ([700, 650, 1, 0, 3], 16, 4, 64, 1)]
    made = []
    for i, (lens, hq, hkv, d, T) in enumerate(shapes):
        c = _int4.make(70 + i, lens, hq, hkv, d, d, 16, T, width=max(640, max(lens)) // 16 + 1)
        call, q, rest = call_of(pkv, c)
        args = (q, *rest, c.lens.cuda(), c.scale)
        made.append((call, args, call(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[] for _ in made]
    for _ in range(40):
        for i, (call, args, _, s) in enumerate(made):
            got[i].append(call(*args, stream=s))
    torch.cuda.synchronize()
    for (_, _, want, _), some in zip(made, got):
        for out, lse in some:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    pkv.device_status()


@pytest.mark.parametrize("d", [128, 96])
def test_a_captured_step_of_a_padded_batch(pkv, d):
    """extend, rotary append and attention in one graph, for a batch whose last rows may be
    padding (length 0, no new token): replayed step by step, it is what the calls one by one
    are, and the padding's blocks and rows stay as they are."""
    B, hq, hkv, bs, width = 6, 8, 2, 16, 48
    g = torch.Generator().manual_seed(d)
    start = [600, 15, 31, 0, 0, 0]

    def state():
        free, pool = pkv.block_pool(B * width)
        tables = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        pools = [torch.full((B * width, hkv, bs, n), fill, dtype=dt, device="cuda")
                 for _ in range(2) for n, dt, fill in ((d // 2, torch.uint8, 255),
                                                       (2, torch.bfloat16, float("nan")))]
        inv = pkv.rope_frequencies(d, device="cuda")
        return free, pool, tables, lens, pools, inv

    def step(s, new, q, k, v):
        free, pool, tables, lens, pools, inv = s
        _, pos, slots = pkv.extend_sequences(tables, lens, new, free, pool, bs, q.shape[0])
        turned = pkv.rope_append_int4(*pools, q, k, v, pos, slots, inv, q_dtype=torch.float32)
        if q.shape[0] != B:
            return None
        return pkv.paged_decode_attn_int4(turned, *pools, tables, lens, d ** -0.5)

    prompt = [torch.randn(sum(start), h, d, generator=g).to(torch.bfloat16).cuda()
              for h in (hq, hkv, hkv)]
    plain, held = state(), state()
    for s in (plain, held):
        step(s, torch.tensor(start, dtype=torch.int32, device="cuda"), *prompt)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        got = step(held, new, q, k, v)
    # (capturing runs nothing)
    for turn in range(20):
        now = [1, 1, 1, int(turn >= 5), int(turn % 3 == 0), 0]
        for t, x in ((new, torch.tensor(now, dtype=torch.int32)),
                     *((t, torch.randn(t.shape, generator=g).to(t.dtype)) for t in (q, k, v))):
            t.copy_(x)
        graph.replay()
        want = step(plain, new.clone(), q.clone(), k.clone(), v.clone())
        torch.cuda.synchronize()
        live = sum(now)
        assert torch.equal(got[1][5], torch.full_like(got[1][5], float("-inf")))
        assert torch.all(got[0][5] == 0)
        # rows of q follow the tokens brought; the others' queries are not written
        assert torch.equal(got[0][:min(live, 3)], want[0][:min(live, 3)])
        for a, b in zip(held[:4], plain[:4]):
            assert torch.equal(a, b)
        for a, b in zip(held[4], plain[4]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert pkv.device_status() == 0
