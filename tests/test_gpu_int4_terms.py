"""Bounds on decode over a 4-bit cache that are tight enough for every term that its sums are
made of: the second terms of query and weights, in both head dims of the tensor-core kernel."""
from __future__ import annotations

import pytest

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


@pytest.mark.parametrize("G,T,kw", [(4, 1, {}), (8, 1, {}), (8, 1, dict(num_splits=1)), (4, 4, {}),
                                    (2, 1, dict(flags=1))])
def test_long_sums_of_small_heads(pkv, G, T, kw):
    """40,000 tokens of nearly equal weights in heads of 64, whose values cancel to a
    two-hundredth: off by 1e-5 of the result at most, as sums in fp32 would be.  (Weights of
    11 bits would be off by 2^-12 of each token's part, 1e-4 of the result.)"""
    c = _int4.make(54, [40000], 2 * G, 2, 64, 64, 64, T, poison=False)
    c.q.mul_(0.05)
    ro = _int4.attend(c)[0]
    out = decode(pkv, c, **kw)[0].cpu().double().view(ro.shape)
    assert float((out - ro).norm() / ro.norm()) < 1e-5


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("G,T", [(4, 1), (8, 1), (4, 4), (16, 1)])
def test_every_term_counts(pkv, G, T, d):
    """A few hundred tokens, against the result's own size.  Errors that are independent from
    token to token add up as the values themselves do, so that the result is off by what one
    token is: 2^-22 by its weight's bits, about 2^-20 by its score (22 bits of the query in a
    sum of terms that is a few times larger), 2^-21 by what sums cut off: 2^-18 leaves room.
    Weights of 11 bits would be off by 2^-12, a query of 11 bits by more."""
    c = _int4.make(55 + G, [300, 77], 2 * G, 2, d, d, 16, T)
    ro, rl, _, _ = _int4.attend(c)
    for kw in (dict(), dict(num_splits=1), dict(num_splits=2)):
        out, lse = decode(pkv, c, **kw)
        out, lse = out.cpu().double().view(ro.shape), lse.cpu().double().view(rl.shape)
        assert float((out - ro).norm() / ro.norm()) < 2.0 ** -18
        assert float((lse - rl).abs().max()) < 2.0 ** -18
