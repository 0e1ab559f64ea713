"""The 4-bit cache on a GPU: append, block copies and decode attention against their
definitions."""
from __future__ import annotations

import math

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


def noise_pools(g, nb, hkv, bs, dk, dv):
    pools = []
    for d in (dk, dv):
        pools += [torch.randint(0, 256, (nb, hkv, bs, d // 2), generator=g).to(torch.uint8),
                  torch.randn(nb, hkv, bs, 2, generator=g).to(torch.bfloat16)]
    return pools


def same_bits(a, b):
    if a.dtype == torch.bfloat16:
        a, b = a.view(torch.int16), b.view(torch.int16)
    return torch.equal(a, b)


def odd_rows(x):
    """Every few rows something a plain row is not: constant, zero, tiny, huge, far from
    zero, infinite, NaN."""
    rows = x.view(-1, x.shape[-1])
    kinds = [lambda r: r.fill_(1.5), lambda r: r.fill_(0.0), lambda r: r.mul_(2.0 ** -130),
             lambda r: r.mul_(2.0 ** -124), lambda r: r.mul_(2.0 ** 120),
             lambda r: r.add_(1000.0), lambda r: r[0:1].fill_(math.inf),
             lambda r: r[-1:].fill_(math.nan), lambda r: r[3:4].fill_(-math.inf),
             lambda r: (r.fill_(3e38), r[1:2].fill_(-3e38)), lambda r: r.fill_(-0.0)]
    for i in range(0, rows.shape[0], 3):
        kinds[(i // 3) % len(kinds)](rows[i])
    return x


@pytest.mark.parametrize("T,hkv,dk,dv,bs", [
    (1, 1, 128, 128, 16), (7, 8, 128, 128, 16), (33, 4, 64, 64, 8), (5, 2, 32, 96, 1),
    (19, 3, 160, 32, 24), (9, 1, 1024, 544, 64), (300, 8, 128, 128, 16), (4, 5, 256, 512, 256)])
def test_append(pkv, T, hkv, dk, dv, bs):
    g = torch.Generator().manual_seed(T)
    nb = -(-T // bs) + 2
    pools = noise_pools(g, nb, hkv, bs, dk, dv)
    k = odd_rows(torch.randn(T, hkv, dk, generator=g).to(torch.bfloat16))
    v = odd_rows(torch.randn(T, hkv, dv, generator=g).to(torch.bfloat16).flip(0))
    slots = torch.randperm(nb * bs, generator=g)[:T].clone()
    if T > 4:
        slots[T // 2] = -1
        slots[1] = nb * bs
    want = [p.clone() for p in pools]
    for x, at in ((k, 0), (v, 2)):
        codes, params = _int4.quantise(x)
        for t in range(T):
            if 0 <= slots[t] < nb * bs:
                b, o = int(slots[t]) // bs, int(slots[t]) % bs
                want[at][b, :, o], want[at + 1][b, :, o] = codes[t], params[t]
    got = [p.cuda() for p in pools]
    pkv.kv_append_int4(*got, k.cuda(), v.cuda(), slots.cuda())
    assert pkv.device_status() == (pkv.DEV_SLOT if T > 4 else 0)
    for i, (a, b) in enumerate(zip(got, want)):
        a = a.cpu()
        if i % 2:                       # a NaN is a NaN
            assert torch.equal(a.isnan(), b.isnan())
            a, b = a.nan_to_num(7.0), b.nan_to_num(7.0)
        assert same_bits(a, b), i


def test_append_of_no_tokens(pkv):
    g = torch.Generator().manual_seed(1)
    got = [p.cuda() for p in noise_pools(g, 2, 2, 16, 128, 128)]
    before = [p.clone() for p in got]
    x = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pkv.kv_append_int4(*got, x, x, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert all(same_bits(a, b) for a, b in zip(got, before)) and pkv.device_status() == 0


@pytest.mark.parametrize("hkv,dk,dv,bs", [(8, 128, 128, 16), (1, 32, 96, 1), (3, 64, 160, 5)])
def test_copy_blocks(pkv, hkv, dk, dv, bs):
    g = torch.Generator().manual_seed(2)
    pools = noise_pools(g, 12, hkv, bs, dk, dv)
    # the fourth pair writes what the fifth reads; the sixth is no block
    src, dst = [0, 1, 0, 5, 6, 12], [9, 10, 11, 6, 7, 3]
    got = [p.cuda() for p in pools]
    pkv.copy_blocks_int4(*got, *(torch.tensor(x, dtype=torch.int32, device="cuda")
                                 for x in (src, dst)))
    assert pkv.device_status() == pkv.DEV_COPY_CONFLICT | pkv.DEV_BLOCK_ID
    for p, a in zip(pools, got):
        want = p.clone()
        for s, d in ((0, 9), (1, 10), (0, 11), (6, 7)):
            want[d] = p[s]
        assert same_bits(a.cpu(), want)


def decode(pkv, c, multi=None, **kw):
    args = (*c.pools(), c.tables.cuda(), c.lens.cuda(), c.scale)
    if c.q.shape[1] > 1 if multi is None else multi:
        return pkv.paged_decode_attn_multi_int4(c.q.cuda(), *args, **kw)
    return pkv.paged_decode_attn_int4(c.q[:, 0].contiguous().cuda(), *args, **kw)


# lens, hq, hkv, dk, dv, bs, tokens
SHAPES = [
    ([1], 1, 1, 128, 128, 16, 1),
    ([0, 5, 16, 17], 8, 2, 128, 128, 16, 1),
    ([31, 32, 33, 64, 65], 4, 4, 128, 128, 8, 1),
    ([300, 1, 127, 128, 129], 32, 8, 128, 128, 16, 1),
    ([257, 1000], 14, 2, 128, 128, 32, 1),
    ([600, 77], 40, 8, 128, 128, 64, 1),
    ([513], 16, 1, 128, 128, 128, 1),
    ([90, 1500], 64, 8, 128, 128, 256, 1),
    ([200, 3], 48, 2, 128, 128, 16, 1),
    ([45, 0, 700], 32, 8, 64, 64, 16, 1),
    ([64, 9], 14, 2, 64, 64, 8, 1),
    ([70, 300], 16, 1, 64, 64, 32, 1),
    ([2, 50, 333], 32, 8, 128, 128, 16, 2),
    ([4, 3, 0, 333], 32, 8, 128, 128, 16, 4),
    ([100, 8], 28, 4, 128, 128, 64, 5),
    ([200], 16, 2, 128, 128, 16, 64),
    ([130, 7], 8, 4, 64, 64, 32, 3),
    # shapes of the CUDA-core kernel
    ([33, 100], 6, 3, 96, 32, 16, 1),
    ([40, 5], 4, 2, 576, 512, 64, 2),
    ([77], 4, 1, 1024, 1024, 3, 1),
    ([130], 8, 2, 128, 64, 16, 2),
    ([130, 40], 8, 2, 128, 128, 12, 2),
    ([50], 2, 1, 256, 256, 4, 1),
]


@pytest.mark.parametrize("lens,hq,hkv,dk,dv,bs,T", SHAPES)
def test_decode(pkv, lens, hq, hkv, dk, dv, bs, T):
    c = _int4.make(len(lens) + hq, lens, hq, hkv, dk, dv, bs, T)
    ref = _int4.attend(c)
    short = pkv.DEV_SEQ_LEN if T > 1 and any(n < T for n in lens) else 0
    for kw in (dict(num_splits=1), dict(num_splits=3), dict(), dict(num_splits=7, flags=1)):
        out, lse = decode(pkv, c, **kw)
        assert pkv.device_status() == short
        _int4.close(out, lse, ref)


@pytest.mark.parametrize("d,G,T", [(128, 4, 1), (128, 8, 1), (128, 4, 4), (64, 4, 1), (96, 2, 1)])
def test_rows_of_very_different_scales(pkv, d, G, T):
    """A token that weighs most may have values of a millionth of the others'."""
    c = _int4.make(3, [700, 90], 2 * G, 2, d, d, 16, T, wide=True)
    ref = _int4.attend(c)
    for kw in (dict(num_splits=1), dict(num_splits=4)):
        _int4.close(*decode(pkv, c, **kw), ref)


@pytest.mark.parametrize("factor", [1e-30, 1e-3, 30.0, 300.0])
def test_queries_of_any_size(pkv, factor):
    c = _int4.make(4, [400, 33], 16, 4, 128, 128, 16)
    c.q.mul_(factor)
    c.q[0, 0, 3] = 0
    _int4.close(*decode(pkv, c), _int4.attend(c))


@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_any_softmax_scale(pkv, scale):
    c = _int4.make(5, [100, 33], 16, 4, 128, 128, 16, scale=scale)
    _int4.close(*decode(pkv, c), _int4.attend(c))


@pytest.mark.parametrize("T,dk", [(1, 128), (4, 128), (1, 96)])
@pytest.mark.parametrize("which", [1, 3])
def test_a_seen_nan_makes_the_row_nan(pkv, which, T, dk):
    c = _int4.make(6, [100, 100], 8, 2, dk, dk, 16, T)
    # the last token of sequence 0: only its last query token sees it
    params = (c.k, c.k_params, c.v, c.v_params)[which]
    params[int(c.tables[0, 6]), :, 3] = math.nan
    ref = _int4.attend(c)
    out, lse = decode(pkv, c, num_splits=2)
    assert out.view(ref[0].shape)[0, -1].isnan().all()
    if which == 1:
        assert lse.view(ref[1].shape)[0, -1].isnan().all()
    keep = torch.ones(ref[1].shape, dtype=torch.bool)
    keep[0, -1] = False
    _int4.close(out.cpu().view(ref[0].shape)[keep], lse.cpu().view(ref[1].shape)[keep],
                [x[keep] for x in ref])


def test_a_nan_query(pkv):
    c = _int4.make(7, [100], 8, 2, 128, 128, 16)
    c.q[0, 0, 1, 5] = math.nan
    c.q[0, 0, 6, 0] = math.inf
    out, lse = decode(pkv, c)
    bad = torch.tensor([False, True, False, False, False, False, True, False])
    assert torch.equal(out.cpu()[0].isnan().all(-1), bad)
    assert torch.equal(lse.cpu()[0].isnan(), bad)


@pytest.mark.parametrize("dk", [128, 96])
def test_bad_pages_and_lengths(pkv, dk):
    c = _int4.make(8, [100, 60, 40], 8, 2, dk, dk, 16)
    ref = _int4.attend(c)
    c.tables[1, 1], c.tables[1, 2] = 1 << 30, -5
    out, lse = decode(pkv, c, num_splits=2)
    assert pkv.device_status() == pkv.DEV_BLOCK_ID
    keep = [0, 2]
    _int4.close(out[keep][:, None], lse[keep][:, None], [x[keep] for x in ref])
    c.tables[1, 1] = c.tables[1, 2] = 0
    c.lens[1] = c.tables.shape[1] * 16 + 1
    out, lse = decode(pkv, c, num_splits=2)
    assert pkv.device_status() == pkv.DEV_SEQ_LEN
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)
    _int4.close(out[keep][:, None], lse[keep][:, None], [x[keep] for x in ref])
    c.lens[1] = -1
    out, lse = decode(pkv, c, num_splits=1)
    assert pkv.device_status() == pkv.DEV_SEQ_LEN and torch.all(out[1] == 0)


@pytest.mark.parametrize("dk,bs", [(128, 16), (96, 16)])
def test_partials_merge_to_the_whole(pkv, dk, bs):
    c = _int4.make(9, [500, 64, 0, 65], 8, 2, dk, dk, bs)
    args = (c.q[:, 0].contiguous().cuda(), *c.pools(), c.tables.cuda(), c.lens.cuda(), c.scale)
    for S in (1, 3, 8):
        op, lp = pkv.paged_decode_attn_partial_int4(*args, S)
        # chunk s of sequence b: 64-token multiples of its length
        for b, L in enumerate(c.lens.tolist()):
            C = 64 * -(-L // (64 * S))
            empty = torch.tensor([s * C >= L for s in range(S)])
            assert torch.equal((lp[:, b, 0] == -math.inf).cpu(), empty)
            assert torch.all(op[empty.cuda(), b] == 0)
        _int4.close(*pkv.lse_merge(op, lp), _int4.attend(c))


def test_repeats_exactly_and_reads_nothing_else(pkv):
    c = _int4.make(10, [3000, 17, 900], 32, 8, 128, 128, 16)
    args = (c.q[:, 0].contiguous().cuda(), *c.pools(), c.tables.cuda(), c.lens.cuda(), c.scale)
    need = pkv.decode_workspace_size_int4(*args[1:5], 3, 32, args[5].shape[1])
    first = pkv.paged_decode_attn_int4(*args)
    for fill in (0, 255):
        ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
        out = torch.full_like(first[0], math.nan)
        again = pkv.paged_decode_attn_int4(*args, workspace=ws, out=out)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert again[0] is out


def test_streams_and_graphs(pkv):
    """Two captured graphs replayed at once on streams of their own."""
    cases = [_int4.make(s, [700, 40], 32, 8, 128, 128, 16, T) for s, T in ((11, 1), (12, 2))]
    held, outs, graphs = [], [], []
    for c in cases:
        q = c.q.cuda() if c.q.shape[1] > 1 else c.q[:, 0].contiguous().cuda()
        call = (pkv.paged_decode_attn_multi_int4 if c.q.shape[1] > 1
                else pkv.paged_decode_attn_int4)
        args = (q, *c.pools(), c.tables.cuda(), c.lens.cuda(), c.scale)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call(*args, stream=s)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            outs.append(call(*args, num_splits=4))
        held.append((args, s))
        graphs.append(graph)
    for _ in range(3):
        for (_, s), graph in zip(held, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cases, outs):
            _int4.close(out, lse, _int4.attend(c))
            out.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("B,longest,hq,hkv,d,bs,T", [
    (40, 900, 32, 8, 128, 16, 1), (3, 6000, 64, 8, 128, 32, 1), (97, 700, 8, 1, 128, 8, 4),
    (33, 1500, 16, 4, 64, 64, 2), (300, 200, 8, 2, 128, 16, 1), (1, 9000, 16, 2, 128, 16, 1),
    (17, 1, 4, 2, 64, 16, 1), (64, 600, 4, 4, 128, 16, 1), (130, 40, 32, 8, 128, 64, 1)])
def test_plans_of_ragged_batches(pkv, B, longest, hq, hkv, d, bs, T):
    """Lengths of every kind, empty ones among them, in tables wide enough for a plan."""
    g = torch.Generator().manual_seed(B + longest)
    lens = torch.randint(0, longest + 1, (B,), generator=g)
    lens[::5] = 0
    lens[-1] = longest
    c = _int4.make(B, lens.tolist(), hq, hkv, d, d, bs, T, width=max(640, longest) // bs + 3)
    out, lse = decode(pkv, c)
    assert pkv.device_status() == (pkv.DEV_SEQ_LEN if T > 1 else 0)
    _int4.close(out, lse, _int4.attend(c))


@pytest.mark.parametrize("B,L,hq,hkv", [(8, 1024, 8, 2), (2, 3000, 8, 8), (1, 5000, 4, 1),
                                        (50, 640, 16, 8), (7, 130, 8, 4)])
def test_plans_of_equal_lengths(pkv, B, L, hq, hkv):
    c = _int4.make(B, [L] * B, hq, hkv, 128, 128, 16, width=max(640, L) // 16 + 1)
    ref = _int4.attend(c)
    out, lse = decode(pkv, c)
    _int4.close(out, lse, ref)
    again = decode(pkv, c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("G,T,kw", [(4, 1, {}), (8, 1, dict(num_splits=1)), (4, 4, {}),
                                    (2, 1, dict(flags=1))])
def test_long_sums_keep_their_precision(pkv, G, T, kw):
    """40,000 tokens of nearly equal weights, whose values cancel to a two-hundredth: off by
    1e-5 of the result at most, as sums in fp32 would be."""
    c = _int4.make(21, [40000], 2 * G, 2, 128, 128, 64, T, poison=False)
    c.q.mul_(0.05)
    ro = _int4.attend(c)[0]
    out = decode(pkv, c, **kw)[0].cpu().double().view(ro.shape)
    assert float((out - ro).norm() / ro.norm()) < 1e-5


@pytest.mark.parametrize("B,Hk,plan", [(160, 8, True), (500, 1, True), (700, 1, False),
                                         (700, 8, False)])
def test_many_pairs(pkv, B, Hk, plan):
    lens = [3 + i % 60 for i in range(B)]
    lens[B // 2] = 700
    c = _int4.make(22, lens, 8, Hk, 64, 64, 8, width=90)
    assert (pkv.decode_workspace_size_int4(*c.pools(), B, 8, 90) > 0) == plan
    _int4.close(*decode(pkv, c), _int4.attend(c))


def test_tables_too_wide_for_the_tensor_cores(pkv):
    """2^30 tokens and more a table row: the CUDA-core kernel numbers them."""
    c = _int4.make(23, [300], 4, 1, 64, 64, 256)
    wide = torch.full((1, (1 << 22) + 1), -1, dtype=torch.int32, device="cuda")
    wide[0, :2] = c.tables[0, :2].cuda()
    out, lse = pkv.paged_decode_attn_int4(c.q[:, 0].contiguous().cuda(), *c.pools(), wide,
                                          c.lens.cuda(), c.scale, num_splits=2)
    _int4.close(out, lse, _int4.attend(c))


def test_far_blocks(pkv):
    """Blocks whose bytes lie past 2^32 in the pool."""
    bs, hkv, d = 16, 8, 128
    nb = (1 << 32) // (bs * hkv * d // 2) + 64
    k = torch.zeros(nb, hkv, bs, d // 2, dtype=torch.uint8, device="cuda")
    kp = torch.zeros(nb, hkv, bs, 2, dtype=torch.bfloat16, device="cuda")
    v, vp = torch.zeros_like(k), torch.zeros_like(kp)
    c = _int4.make(13, [100, 333], 32, 8, d, d, bs, poison=False)
    far = c.tables.clone()
    for b in range(2):
        for i in range(far.shape[1]):
            if c.tables[b, i] >= 0:
                src, to = int(c.tables[b, i]), nb - 1 - int(c.tables[b, i])
                for pool, x in ((k, c.k), (kp, c.k_params), (v, c.v), (vp, c.v_params)):
                    pool[to] = x[src].cuda()
                far[b, i] = to
    ref = _int4.attend(c)
    for flags in (0, 1):
        out, lse = pkv.paged_decode_attn_int4(c.q[:, 0].contiguous().cuda(), k, kp, v, vp,
                                              far.cuda(), c.lens.cuda(), c.scale, flags=flags)
        _int4.close(out, lse, ref)
    x = torch.randn(3, hkv, d).to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 1, nb * bs - 40, nb * bs - 33])
    pkv.kv_append_int4(k, kp, v, vp, x.cuda(), x.cuda(), slots.cuda())
    codes, params = _int4.quantise(x)
    for t, slot in enumerate(slots.tolist()):
        assert same_bits(v[slot // bs, :, slot % bs].cpu(), codes[t])
        assert same_bits(vp[slot // bs, :, slot % bs].cpu(), params[t])
    assert pkv.device_status() == 0


# lens, hq, hkv, dk, dv, bs, tokens: rows of one to four words a lane, of 8, 16 and 32 lanes;
# one to nine query heads a KV head
@pytest.mark.parametrize("lens,hq,hkv,dk,dv,bs,T", [
    ([0, 1, 2, 31], 3, 3, 32, 32, 1, 1), ([65, 64, 200], 10, 2, 64, 32, 5, 1),
    ([3, 129, 17], 9, 3, 96, 128, 24, 3), ([300, 7], 9, 1, 160, 64, 256, 1),
    ([33, 5, 400], 4, 2, 224, 256, 16, 2), ([70, 130], 6, 2, 288, 96, 32, 1),
    ([40, 1, 0, 90], 2, 2, 512, 544, 16, 4), ([150], 7, 1, 1024, 32, 16, 1),
    ([1, 640, 63], 14, 2, 128, 128, 16, 5), ([500, 12], 8, 8, 64, 64, 8, 1)])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_cuda_core_shapes(pkv, lens, hq, hkv, dk, dv, bs, T, splits):
    c = _int4.make(31 + hq + T, lens, hq, hkv, dk, dv, bs, T)
    got = decode(pkv, c, num_splits=splits, flags=pkv.DECODE_GENERIC)
    _int4.close(*got, _int4.attend(c))
    pkv.device_status()


def test_lengths_written_just_before(pkv):
    """Steps that follow one another without a pause, their lengths written by the kernel
    before (a copy; an extend): the plan and the merge both go by the new ones."""
    c = _int4.make(41, [2500, 700, 1300, 3000, 90], 8, 2, 128, 128, 16, width=190)
    args = (c.q[:, 0].contiguous().cuda(), *c.pools(), c.tables.cuda())
    sets = [c.lens.cuda(), torch.tensor([40, 700, 1100, 129, 90], dtype=torch.int32).cuda(),
            torch.tensor([2500, 0, 1, 2999, 60], dtype=torch.int32).cuda()]
    want = []
    for lens in sets:
        want.append(pkv.paged_decode_attn_int4(*args, lens, c.scale))
        torch.cuda.synchronize()
    now, got = sets[0].clone(), []
    for i in range(60):
        now.copy_(sets[i % 3])
        got.append(pkv.paged_decode_attn_int4(*args, now, c.scale))
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    # the tables hold more blocks than the lengths need: an extend within them takes none
    tables, lens = args[-1].clone(), sets[1].clone()
    free, state = pkv.block_pool(c.k.shape[0], args[0].device)
    state[0] = 0
    one = torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
    lens.copy_(torch.tensor([33, 700, 1090, 129, 81], dtype=torch.int32))
    got = []
    for i in range(5):
        pkv.extend_sequences(tables, lens, one, free, state, 16, 8)
        got.append(pkv.paged_decode_attn_int4(*args, lens, c.scale))
    for i in range(5):
        at = torch.tensor([34 + i, 700, 1091 + i, 129, 82 + i], dtype=torch.int32, device="cuda")
        out, lse = pkv.paged_decode_attn_int4(*args, at, c.scale)
        assert torch.equal(out, got[i][0]) and torch.equal(lse, got[i][1])
    assert pkv.device_status() == 0
