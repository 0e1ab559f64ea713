"""Block tables on the GPU at the largest batches: prefix sums past 48 KB of shared memory, five
and more sequences a thread, one CTA and several; and extends and trims of two pools at once."""
from __future__ import annotations

import random

import pytest
import torch

from tests.test_gpu_tables import Plain, check, extend, trim

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_93_gb300 as m
    m.device_status(reset=True)
    return m


# at most 4,096 rows: one CTA; more: several
@pytest.mark.parametrize("B,most_new", [(4095, 1), (4096, 1), (4097, 1), (4096, 3), (5000, 2),
                                        (8191, 2), (8192, 1), (8192, 4)])
def test_steps(pkv, B, most_new):
    rng = random.Random(B + most_new)
    bs = 4
    lens = [rng.randint(0, 6) for _ in range(B)]
    nb = sum(-(-n // bs) for n in lens) + 2 * B + 9
    plain = Plain(lens, 5, bs, nb, rng)
    t = plain.tensors()
    for turn in range(2):
        new = [rng.choice([0, rng.randint(1, most_new)]) for _ in range(B)]
        if B > 4096:
            new[-1] = 1
        extend(pkv, t, plain, new, sum(new) + rng.choice([0, 1, 13]))
        trim(pkv, t, plain, [rng.choice([-1, n, rng.randint(0, n)]) for n in plain.lens])


@pytest.mark.parametrize("B", [4096, 8192])
@pytest.mark.parametrize("blocks,rows", [(1.0, 0.5), (0.4, 1.0), (0.3, 0.6), (0.0, 1.0)])
def test_what_does_not_fit_is_refused(pkv, B, blocks, rows):
    rng = random.Random(B)
    bs = 4
    lens = [rng.randint(0, 8) for _ in range(B)]
    new = [rng.choice([0, 1, 3, 9, 30]) for _ in range(B)]
    need = sum(-(-(a + n) // bs) - -(-a // bs) for a, n in zip(lens, new) if a + n <= 5 * bs)
    plain = Plain(lens, 5, bs, sum(-(-n // bs) for n in lens) + need + 5, rng, int(blocks * need))
    t = plain.tensors()
    extend(pkv, t, plain, new, int(rows * sum(new)))
    trim(pkv, t, plain, [rng.choice([-1, 0, n]) for n in plain.lens])


def test_two_pools_at_once(pkv):
    """Extends and trims of two states in flight on two streams."""
    rng = random.Random(9)
    made = []
    for B, most in ((300, 40), (2000, 5)):
        plain = Plain([rng.randint(0, 90) for _ in range(B)], 60, 16, 60 * B, rng)
        made.append((plain, plain.tensors(), torch.cuda.Stream(), most))
    torch.cuda.synchronize()
    for turn in range(6):
        wants = []
        for plain, t, s, most in made:
            new = [rng.randint(0, most) for _ in plain.lens]
            rows = sum(new) + 3
            cu, positions, slots, flags = plain.extend(new, rows, pkv)
            keep = [max(0, n - rng.randint(0, 3)) for n in plain.lens]
            assert flags == plain.trim(keep, pkv) == 0
            with torch.cuda.stream(s):
                args = [torch.tensor(x, dtype=torch.int32).pin_memory().to("cuda",
                                                                          non_blocking=True)
                        for x in (new, keep)]
            got = pkv.extend_sequences(t["tables"], t["lens"], args[0], t["free"], t["state"], 16,
                                       rows, stream=s)
            pkv.trim_sequences(t["tables"], t["lens"], args[1], t["free"], t["state"], 16,
                               stream=s)
            wants.append((got, (cu, positions, slots), args))
        torch.cuda.synchronize()
        for got, want, _ in wants:
            for a, b in zip(got, want):
                assert a.tolist() == b
        for plain, t, _, _ in made:
            check(t, plain)
    assert pkv.device_status() == 0
