"""The binding of the 4-bit cache's calls: numbers past 32 bits.  Every call here is refused by
its arguments; nothing reaches a GPU."""
from __future__ import annotations

import pytest
import torch

from tests import _int4
from tests.test_int4_host import cpu, pkv  # noqa: F401  (fixtures)


def test_numbers_past_32_bits_do_not_wrap_around(cpu):  # noqa: F811
    c = _int4.make(1, [20, 3], 8, 2, 128, 128, 16)
    pools = (c.k, c.k_params, c.v, c.v_params)
    size = cpu.decode_workspace_size_int4
    big = 2 ** 32
    assert size(*pools, 2, 8, 4, num_splits=3) > 0
    assert size(*pools, big + 2, 8, 4, num_splits=3) == 0
    assert size(*pools, 2, 8, 4, tokens_per_seq=big + 1, num_splits=3) == 0
    assert size(*pools, 2, big + 8, 4, num_splits=3) == 0
    assert size(*pools, 2, 8, -big, num_splits=3) == 0
    q = c.q[:, 0].contiguous()
    rest = (*pools, c.tables, c.lens, 0.1)
    for flags in (big, -big, big + 1):
        for call in (lambda: cpu.paged_decode_attn_int4(q, *rest, num_splits=1, flags=flags),
                     lambda: cpu.paged_decode_attn_multi_int4(c.q, *rest, num_splits=1,
                                                              flags=flags),
                     lambda: cpu.paged_decode_attn_partial_int4(
                         q, *rest, 1, torch.empty(1, 2, 8, 128), torch.empty(1, 2, 8),
                         flags=flags)):
            with pytest.raises(cpu.PkvError) as e:
                call()
            assert e.value.status == -1
