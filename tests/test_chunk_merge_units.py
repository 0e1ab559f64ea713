"""How the merge's warps walk its work, at the limits of a call, on the CPU: the
header the kernel uses, compiled for the host, against 64-bit arithmetic."""
from __future__ import annotations

import os
import subprocess

import pytest

from tests.conftest import ROOT

SRC = r"""
#include <cstdio>
#include <cstdlib>
#include "chunk_merge_units.h"
int main(int, char **v) {
    const int32_t entries = atoi(v[1]), units = atoi(v[2]), rest = atoi(v[3]);
    const int32_t stride = atoi(v[4]), first = atoi(v[5]);
    const int64_t own = (int64_t)entries * units, total = own + rest;
    int64_t w = first;
    for (pkv::MergeWalk m(first, stride, entries, units, rest); !m.done(); m.next(), w += stride) {
        const bool in = w < own;
        if (w >= total || m.in_entries() != in) return 2;
        if (in ? (m.unit != w / entries || m.entry != w % entries) : (m.piece() != w - own)) return 3;
    }
    return w < total ? 4 : 0;             // it stopped where the work ends
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    (d / "units.cpp").write_text(SRC)
    csrc = os.path.join(ROOT, "paged_kv_cache_93_gb300", "csrc")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", csrc, str(d / "units.cpp"),
                           "-o", str(d / "units")])
    return str(d / "units")


# (entries, units): none; a few; 65,535 sequences over 1,025 KV heads, one of them with
# 128 rows (2^31 pieces and more); as many query rows as a call may have
@pytest.mark.parametrize("entries,units", [(0, 0), (0, 32), (1, 1), (7, 1), (24 * 8, 32),
                                           (65535 * 1025, 32), ((1 << 29) - 1, 32),
                                           ((1 << 29) - 1, 1)])
@pytest.mark.parametrize("rest", [0, 64, 256 * 64])
def test_every_piece_once(program, entries, units, rest):
    for stride in (8, 9728):
        if entries * units // stride > 10 ** 8:
            continue
        for first in (0, 1, stride - 1):
            assert subprocess.call([program, *map(str, (entries, units, rest, stride, first))]) == 0
