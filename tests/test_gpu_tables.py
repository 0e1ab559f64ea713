"""Block tables and slot maps kept on the GPU (extend_sequences, trim_sequences) against
the same steps taken one sequence at a time."""
from __future__ import annotations

import random

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


class Plain:
    """The documented rules, one sequence after another."""

    def __init__(self, lens, width, bs, num_blocks, rng, free=None):
        self.bs, self.nb, self.width = bs, num_blocks, width
        order = list(range(num_blocks))
        rng.shuffle(order)
        self.tables = [[rng.randint(-3, 3) for _ in range(width)] for _ in lens]
        for row, n in zip(self.tables, lens):
            for i in range(-(-n // bs)):
                row[i] = order.pop()
        self.free, self.count = order + [0] * (num_blocks - len(order)), len(order)
        if free is not None:
            self.count = min(self.count, free)
        self.lens = list(lens)

    def tensors(self):
        t = {n: torch.tensor(x, dtype=torch.int32, device="cuda")
             for n, x in (("tables", self.tables), ("lens", self.lens), ("free", self.free),
                          ("state", [self.count, 0, 0, 0]))}
        t["tables"] = t["tables"].view(len(self.lens), self.width)
        return t

    def extend(self, new, rows, pkv):
        flags = asked_rows = asked_blocks = at = 0
        most = self.width * self.bs
        cu, positions, slots = [0], [], []
        for b, n in enumerate(new):
            old, ok = self.lens[b], True
            if n < 0 or not 0 <= old <= most:
                flags, ok = flags | pkv.DEV_SEQ_LEN, False
            elif old + n > most:
                flags, ok = flags | pkv.DEV_TABLE_RANGE, False
            need = 0
            if ok:
                asked_rows += n
                if n > 0 and asked_rows > rows:
                    flags, ok = flags | pkv.DEV_QUERY_RANGE, False
            if ok:
                need = -(-(old + n) // self.bs) + -old // self.bs
                asked_blocks += need
                if need > 0 and asked_blocks > self.count + at:
                    flags, ok = flags | pkv.DEV_NO_BLOCKS, False
            if not ok:
                n = need = 0
            for i in range(need):
                self.count -= 1
                at += 1
                self.tables[b][-(-old // self.bs) + i] = self.free[self.count]
            for p in range(old, old + n):
                phys = self.tables[b][p // self.bs]
                positions.append(p)
                slots.append(phys * self.bs + p % self.bs)
            self.lens[b] += n
            cu.append(len(positions))
        pad = [-1] * (rows - len(positions))
        return cu, positions + pad, slots + pad, flags

    def trim(self, keep, pkv):
        flags = 0
        for b in reversed(range(len(keep))):
            k, old = keep[b], self.lens[b]
            if k < 0:
                continue
            if k > old or not 0 <= old <= self.width * self.bs:
                flags |= pkv.DEV_SEQ_LEN
                continue
            for i in reversed(range(-(-k // self.bs), -(-old // self.bs))):
                self.free[self.count] = self.tables[b][i]
                self.count += 1
            self.lens[b] = k
        return flags


def check(t, plain):
    assert t["tables"].tolist() == plain.tables
    assert t["lens"].tolist() == plain.lens
    assert t["state"].tolist() == [plain.count, 0, 0, 0]
    assert t["free"].tolist()[:plain.count] == plain.free[:plain.count]


def extend(pkv, t, plain, new, rows):
    cu, positions, slots, flags = plain.extend(new, rows, pkv)
    got = pkv.extend_sequences(t["tables"], t["lens"],
                               torch.tensor(new, dtype=torch.int32, device="cuda"), t["free"],
                               t["state"], plain.bs, rows)
    assert pkv.device_status() == flags
    for a, b in zip(got, (cu, positions, slots)):
        assert a.tolist() == b
    check(t, plain)


def trim(pkv, t, plain, keep):
    flags = plain.trim(keep, pkv)
    pkv.trim_sequences(t["tables"], t["lens"],
                       torch.tensor(keep, dtype=torch.int32, device="cuda"), t["free"],
                       t["state"], plain.bs)
    assert pkv.device_status() == flags
    check(t, plain)


@pytest.mark.parametrize("B,longest,most_new,bs", [
    (1, 0, 1, 16), (1, 100, 70, 16), (3, 40, 5, 1), (33, 300, 9, 7), (256, 500, 1, 16),
    (300, 50, 100, 256), (513, 100, 3, 64), (1000, 64, 30, 16), (2049, 8, 4, 2)])
def test_steps(pkv, B, longest, most_new, bs):
    rng = random.Random(B)
    lens = [rng.randint(0, longest) for _ in range(B)]
    width = -(-(longest + 3 * most_new) // bs) + 1
    nb = sum(-(-n // bs) for n in lens) + B * (-(-3 * most_new // bs) + 1)
    plain = Plain(lens, width, bs, nb, rng)
    t = plain.tensors()
    for step in range(3):
        new = [rng.choice([0, rng.randint(1, most_new)]) for _ in range(B)]
        extend(pkv, t, plain, new, sum(new) + rng.choice([0, 1, 13]))
        keep = [rng.choice([-1, n, rng.randint(0, n), 0 if rng.random() < 0.1 else n])
                for n in plain.lens]
        trim(pkv, t, plain, keep)


@pytest.mark.parametrize("B", [1, 5, 600])
def test_what_does_not_fit_is_refused(pkv, B):
    rng = random.Random(100 + B)
    bs = 8
    for free, rows in ((B, 10 ** 6), (10 ** 6, 3 * B), (B // 2, 2 * B), (0, 0), (1, 7)):
        lens = [rng.randint(0, 60) for _ in range(B)]
        plain = Plain(lens, 12, bs, sum(-(-n // bs) for n in lens) + 4 * B + 8, rng, free)
        if B > 1:
            plain.lens[1] = 97
            plain.lens[2] = -1
        t = plain.tensors()
        new = [rng.choice([0, 1, 5, 20, 50, -1]) for _ in range(B)]
        extend(pkv, t, plain, new, min(rows, sum(max(0, n) for n in new) + 5))
        # (the stray lengths hold no blocks)
        trim(pkv, t, plain, [rng.choice([-1, 200, 0, 5]) for _ in range(B)])


def test_trim_to_the_old_lengths_undoes_an_extend(pkv):
    rng = random.Random(3)
    plain = Plain([rng.randint(0, 900) for _ in range(700)], 80, 16, 60000, rng)
    t = plain.tensors()
    before = {n: x.clone() for n, x in t.items()}
    new = torch.tensor([rng.randint(0, 300) for _ in range(700)], dtype=torch.int32, device="cuda")
    for _ in range(3):
        pkv.extend_sequences(t["tables"], t["lens"], new, t["free"], t["state"], 16, 120000)
        assert not torch.equal(t["lens"], before["lens"])
        pkv.trim_sequences(t["tables"], t["lens"], before["lens"], t["free"], t["state"], 16)
        for n in ("lens", "free", "state"):
            assert torch.equal(t[n], before[n]), n
    assert pkv.device_status() == 0


def test_one_long_sequence_comes_and_goes(pkv):
    rng = random.Random(4)
    plain = Plain([0, 5], 12501, 16, 12600, rng)
    t = plain.tensors()
    extend(pkv, t, plain, [200000, 1], 200001)
    trim(pkv, t, plain, [0, -1])


def test_bad_blocks_and_counts_are_told(pkv):
    rng = random.Random(5)
    plain = Plain([20, 3], 6, 16, 30, rng)
    t = plain.tensors()
    t["free"][plain.count - 1] = 30             # the first block taken
    t["tables"][1, 0] = -7
    new = torch.tensor([20, 2], dtype=torch.int32, device="cuda")
    _, positions, slots = pkv.extend_sequences(t["tables"], t["lens"], new, t["free"],
                                               t["state"], 16, 22)
    assert pkv.device_status() == pkv.DEV_BLOCK_ID
    assert positions.tolist() == [*range(20, 40), 3, 4]
    # positions 20 to 31 lie in a block that was there, 32 to 39 in the bad one
    assert all(s >= 0 for s in slots.tolist()[:12]) and slots.tolist()[12:] == [-1] * 10
    assert t["tables"][0, 2] == 30
    for count in (-1, 31):
        t["state"][0] = count
        _, positions, _ = pkv.extend_sequences(t["tables"], t["lens"], new * 10, t["free"],
                                               t["state"], 16, 300)
        assert pkv.device_status() & pkv.DEV_BLOCK_ID
        assert t["state"].tolist() == [0, 0, 0, 0]
    # more blocks than the stack has room for
    t["state"][0] = 29
    pkv.trim_sequences(t["tables"], t["lens"], torch.zeros_like(t["lens"]), t["free"],
                       t["state"], 16)
    assert pkv.device_status() == pkv.DEV_BLOCK_ID and t["state"].tolist() == [30, 0, 0, 0]


def test_no_sequences(pkv):
    free, state = pkv.block_pool(4)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu, positions, slots = pkv.extend_sequences(e.view(0, 3), e, e, free, state, 16, 5)
    assert cu.tolist() == [0] and positions.tolist() == slots.tolist() == [-1] * 5
    pkv.trim_sequences(e.view(0, 3), e, e, free, state, 16)
    assert state.tolist() == [4, 0, 0, 0] and free.tolist() == [3, 2, 1, 0]
    assert pkv.device_status() == 0


def test_in_a_graph(pkv):
    rng = random.Random(6)
    plain = Plain([rng.randint(0, 90) for _ in range(64)], 40, 16, 3000, rng)
    t = plain.tensors()
    new = torch.zeros(64, dtype=torch.int32, device="cuda")
    keep = torch.zeros(64, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    args = (t["free"], t["state"], 16)
    rows = 64 * 40
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = pkv.extend_sequences(t["tables"], t["lens"], new, *args, rows)
        pkv.trim_sequences(t["tables"], t["lens"], keep, *args)
    for _ in range(4):
        n = [rng.randint(0, 40) for _ in range(64)]
        k = [max(0, a + b - rng.randint(0, 5)) for a, b in zip(plain.lens, n)]
        new.copy_(torch.tensor(n))
        keep.copy_(torch.tensor(k))
        cu, positions, slots, flags = plain.extend(n, rows, pkv)
        flags |= plain.trim(k, pkv)
        torch.cuda.synchronize()
        graph.replay()
        assert pkv.device_status() == flags == 0
        for a, b in zip(got, (cu, positions, slots)):
            assert a.tolist() == b
        check(t, plain)
