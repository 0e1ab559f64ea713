"""Decode over a 4-bit cache where its sums have least room: value rows that are constant
(scale 0, the offset alone), offsets of any size, scores that rise, very long sequences."""
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


def decode(pkv, c, **kw):
    args = (*c.pools(), c.tables.cuda(), c.lens.cuda(), c.scale)
    if c.q.shape[1] > 1:
        return pkv.paged_decode_attn_multi_int4(c.q.cuda(), *args, **kw)
    return pkv.paged_decode_attn_int4(c.q[:, 0].contiguous().cuda(), *args, **kw)


def constant_rows(c, codes, params, at, values):
    """Rows `at` [n] of sequence 0, every head's, become constant rows of values [n]: codes 0,
    scale 0, the value as offset, as the append stores them."""
    bs = c.k.shape[2]
    block, place = c.tables[0, at // bs].long(), at % bs
    row = torch.stack((torch.zeros(len(at)), values), -1).to(torch.bfloat16)
    codes[block, :, place] = 0
    params[block, :, place] = row[:, None]


# query rows of a KV head: 4, 8 and 16
@pytest.mark.parametrize("G,T", [(4, 1), (8, 1), (4, 4)])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("value", [0.0, 1000.0, 2.0 ** 28, -2.0 ** 100])
def test_constant_values_under_rising_scores(pkv, value, d, G, T):
    """Every value row is constant and the scores rise by nearly 10 base-2 units after each
    warp's first tile: the result is the constant."""
    L = 9000
    c = _int4.make(51, [L], 2 * G, 2, d, d, 64, T)
    j = torch.arange(L)
    # a warp of the four of num_splits=1 has 71 tiles of 32 tokens
    high = j % (71 * 32) >= 32
    constant_rows(c, c.k, c.k_params, j, torch.where(high, 6.8125, 0.0))  # 9.83 base-2 units
    constant_rows(c, c.v, c.v_params, j, torch.full((L,), value))
    h = torch.arange(2 * G)[:, None]
    c.q = ((1 - 0.01 * h) / (c.scale * d)).expand(1, T, 2 * G, d).contiguous()
    ref = _int4.attend(c)
    for kw in (dict(), dict(num_splits=1), dict(num_splits=3), dict(flags=pkv.DECODE_GENERIC)):
        _int4.close(*decode(pkv, c, **kw), ref)
    assert pkv.device_status() == 0


@pytest.mark.parametrize("G,T,d", [(4, 1, 128), (8, 1, 128), (4, 4, 128), (4, 1, 64), (8, 1, 64),
                                   (4, 4, 64)])
@pytest.mark.parametrize("first,then", [(0.0, 2.0 ** 60), (2.0 ** -60, 2.0 ** 60),
                                        (1.0, -2.0 ** 80), (2.0 ** 90, 2.0 ** -90)])
def test_constant_values_of_mixed_sizes(pkv, first, then, G, T, d):
    """Constant rows of one size, then of another, a few ordinary ones between: the larger ones
    may come when the reference has long been settled."""
    L = 3000
    c = _int4.make(52, [L], 2 * G, 2, d, d, 64, T)
    j = torch.arange(L)
    plain = j % 50 == 7
    values = torch.where(j < 1700, first, then) * (1 + (j % 4) / 4)
    constant_rows(c, c.v, c.v_params, j[~plain], values[~plain])
    ref = _int4.attend(c)
    for kw in (dict(), dict(num_splits=1), dict(flags=pkv.DECODE_GENERIC)):
        _int4.close(*decode(pkv, c, **kw), ref)


@pytest.mark.parametrize("G,d", [(4, 128), (8, 128), (16, 128), (4, 64), (8, 64), (16, 64)])
def test_constant_rows_keep_the_scores_bits(pkv, G, d):
    """Two tokens of values 1 and -1 and nearly equal scores.  With p the weights, a relative
    error of each by r moves the result by 2 p1 p2 (2 r) <= r.  The scores are within 2^-3 of 0
    and their products within 2^-22 of what they are; held 15 base-2 units above the
    reference they are rounded twice by half a step of 2^-20 (the sum with the key's offset,
    the sum with the scale's product), and the exponential is off by 2^-22: r is at most
    ln 2 (2 * 2^-21 + 2^-22) + 2^-22 < 2^-20 + 2^-23.  Held 100 units above, it would be 8
    times that."""
    B = 64
    c = _int4.make(53, [2] * B, 2 * G, 2, d, d, 16)
    c.q.mul_(0.002)
    for b in range(B):
        block = int(c.tables[b, 0])
        c.v[block, :, :2] = 0
        c.v_params[block, :, 0] = torch.tensor([0.0, 1.0], dtype=torch.bfloat16)
        c.v_params[block, :, 1] = torch.tensor([0.0, -1.0], dtype=torch.bfloat16)
    ro = _int4.attend(c)[0]
    for kw in (dict(), dict(num_splits=1)):
        out = decode(pkv, c, **kw)[0].cpu().double().view(ro.shape)
        assert float((out - ro).abs().max()) <= 2.0 ** -20 + 2.0 ** -23


@pytest.mark.parametrize("value", [0.0, 1.0])
@pytest.mark.parametrize("G,d", [(4, 128), (16, 64)])
def test_the_weights_of_many_million_tokens(pkv, G, d, value):
    """9 million tokens (a few blocks, again and again), the same in all but the first tile of
    each warp, whose scores are lower by 7.89 base-2 units.  The sum of weights has room for
    all of them; lse by arithmetic."""
    bs, blocks = 256, 36000
    L = bs * blocks
    zero = torch.zeros(2, 1, bs, d // 2, dtype=torch.uint8, device="cuda")
    k_params = torch.zeros(2, 1, bs, 2, dtype=torch.bfloat16, device="cuda")
    v_params = torch.zeros_like(k_params)
    k_params[1, :, :, 1] = 5.46875
    v_params[..., 1] = value
    tables = torch.ones(1, blocks, dtype=torch.int32, device="cuda")
    tables[0, ::blocks // 4] = 0                # a warp's first block, low
    q = torch.full((1, G, d), 1.0 / d, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_decode_attn_int4(q, zero, k_params, zero, v_params, tables, lens, 1.0,
                                          num_splits=1)
    want = math.log(4 * bs + (L - 4 * bs) * math.exp(5.46875))
    assert pkv.device_status() == 0
    # lse: 72,000 tiles' sums in a chain a lane, each off by half a step at most, 72,000 * 2^-24
    # of the sum together; scores and the result itself round by 2^-20 and less
    assert float((lse.double() - want).abs().max()) < 72000 * 2.0 ** -24 + 2.0 ** -18
    # out: the same sums above and below the line
    assert float((out.double() - value).abs().max()) <= 2.0 ** -18 * value


@pytest.mark.parametrize("G,T,d", [(4, 1, 128), (8, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -90, 2.0 ** -30, 2.0 ** 30, 2.0 ** 90])
def test_values_of_unusual_sizes(pkv, size, G, T, d):
    """Weights and lse within 2^-17 where all values are tiny, huge or zero; and what the
    products' 22 bits and the scores' sums add, as elsewhere (2^-18 each)."""
    c = _int4.make(56, [300, 5, 40], 2 * G, 2, d, d, 16, T)
    c.v_params = (c.v_params.float() * size).to(torch.bfloat16)
    c.q.mul_(0.1)
    ro, rl, tol, _ = _int4.attend(c)
    for kw in (dict(), dict(num_splits=2)):
        out, lse = decode(pkv, c, **kw)
        out, lse = out.cpu().double().view(ro.shape), lse.cpu().double().view(rl.shape)
        # (tol is 2^-18 of the sum of weights times values' sizes, and more)
        assert torch.all((out - ro).abs() <= 3 * tol)
        assert float((lse - rl).abs().max()) <= 2.0 ** -17 + 2.0 ** -18
    assert pkv.device_status() == 0
