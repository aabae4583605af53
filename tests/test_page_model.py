"""The plain model of the page calls keeps what must always hold (counts are the table's
references, no page written by two sequences), so that the GPU calls may be held to it."""
from __future__ import annotations

import random

import pytest

from page_model import Pages


def check(m: Pages):
    count = [0] * m.num_pages
    for row in m.rows:
        for x in row:
            if x >= 0:
                count[x] += 1
    assert count == m.refs
    for b in range(m.B):
        full = m.lens[b] // m.P
        for x in m.rows[b][full:]:  # pages that appends write to
            assert x < 0 or count[x] == 1


@pytest.mark.parametrize("seed", range(6))
def test_random_calls_keep_the_invariants(seed):
    rng = random.Random(seed)
    B, P, maxp = rng.choice([(1, 64, 3), (5, 64, 4), (9, 128, 3)])
    m = Pages(B, maxp, rng.choice([B * maxp, B * maxp // 2 + 1]), P)
    for _ in range(200):
        op = rng.randrange(4)
        if op == 0:
            m.reserve([rng.choice([0, 1, 30, 200]) for _ in range(B)])
        elif op == 1:
            for b in range(B):  # append into reserved pages
                held = next((j for j, x in enumerate(m.rows[b]) if x < 0), maxp) * P
                m.lens[b] = max(m.lens[b], rng.randrange(m.lens[b], held + 1) if held >= m.lens[b] else 0)
        elif op == 2:
            m.reorder([rng.choice([b, b, rng.randrange(-1, B)]) for b in range(B)])
        else:
            new = m.compact()
            live = sorted(x for x in new if x >= 0)
            assert live == list(range(len(live)))
        check(m)


def test_fork_and_free_by_hand():
    m = Pages(3, 4, 8, 64)
    m.reserve([200, 0, 64])
    assert m.rows[0] == [0, 1, 2, 3] and m.rows[2] == [4, -1, -1, -1] and m.info == [5, 0, 5, 0]
    m.lens = [130, 0, 64]
    assert m.reorder([0, 0, -1]) == [(1, 0, 2, 4)]  # page 4 of sequence 2 is free at once
    assert m.rows[1] == [0, 1, 4, -1] and m.refs == [2, 2, 1, 1, 1, 0, 0, 0] and m.lens == [130, 130, 0]
    assert m.info == [1, 0, 5, 1]
    m.reorder([-1, 1, 2])
    assert m.refs == [1, 1, 0, 0, 1, 0, 0, 0]
    assert m.compact() == [0, 1, -1, -1, 2, -1, -1, -1] and m.rows[1] == [0, 1, 2, -1]
