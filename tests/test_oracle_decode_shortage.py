"""Forks that run out of pages or of room in the tables: a page that a sequence
still holds is never written for another one (CPU)."""

import numpy as np
import pytest

from oracle import decode

I = np.int32   # noqa: E741


def test_a_page_whose_other_holder_found_no_page_is_not_kept():
    # both sequences have 20 tokens and share page 1; no page is free
    tables, lens, refs = np.array([[0, 1], [0, 1]], I), np.array([20, 20], I), np.array([2, 2], I)
    t, n, r, s = decode.fork(tables, lens, refs, 16, None, [1, 1])
    assert n.tolist() == [20, 20] and np.array_equal(t, tables) and np.array_equal(r, refs) and s.tolist() == [0, 1, 2, 0]
    # with one free page the first copies, the second keeps
    t, n, r, s = decode.fork(tables, lens, np.array([2, 2, 0], I), 16, None, [1, 1])
    assert n.tolist() == [21, 21] and t.tolist() == [[0, 2], [0, 1]] and r.tolist() == [2, 1, 1] and s.tolist() == [0, 0, 0, 1]
    # three of them and one free page: the second is short of a copy, so the third may not keep the page
    t, n, r, s = decode.fork(tables, lens, np.array([2, 2, 0], I), 16, [0, 0, 1], [1, 1, 1])
    assert n.tolist() == [21, 20, 20] and t.tolist() == [[0, 2], [0, 1], [0, 1]] and r.tolist() == [3, 2, 1]
    assert s.tolist() == [0, 1, 2, 1]


def test_a_page_whose_other_holder_has_no_room_is_copied():
    # sequence 0 asks for more than its table has room for and stays in page 1; sequence 1 would write there
    tables, lens, refs = np.array([[0, 1], [0, 1]], I), np.array([25, 20], I), np.array([2, 2, 0], I)
    t, n, r, s = decode.fork(tables, lens, refs, 16, None, [100, 1])
    assert n.tolist() == [25, 21] and t.tolist() == [[0, 1], [0, 2]] and r.tolist() == [2, 1, 1] and s.tolist() == [0, 0, 1, 1]
    t, n, r, s = decode.fork(tables, lens, refs, 16, [1, 0], [1, 100])      # whichever comes first
    assert n.tolist() == [21, 25] and t.tolist() == [[0, 2], [0, 1]] and r.tolist() == [2, 1, 1] and s.tolist() == [0, 0, 1, 1]
    t, n, r, s = decode.fork(tables, lens, refs[:2], 16, None, [100, 1])
    assert n.tolist() == [25, 20] and np.array_equal(t, tables) and r.tolist() == [2, 2] and s.tolist() == [0, 1, 2, 0]


@pytest.mark.parametrize("most", [9, 45])
@pytest.mark.parametrize("seed", [*range(60), 212])
def test_every_sequence_keeps_its_tokens(seed, most):
    """What each sequence holds is what was written for it, in pools of which most steps are short."""
    rng = np.random.default_rng(seed)
    page, M, P, n, missed = 16, 3, int(rng.integers(1, 9)), 5, 0
    tables, lens, refs = np.full((n, M), -1, I), np.zeros(n, I), np.zeros(P, I)
    texts, pool = [[] for _ in range(n)], np.zeros((P, page), I)
    for _ in range(40):
        m = int(rng.integers(1, 8))
        parents, grow = rng.integers(-1, n, size=m), rng.integers(0, most, size=m)
        old = lens
        tables, lens, refs, state = decode.fork(tables, lens, refs, page, parents, grow, [pool])
        texts = [list(texts[p]) if p >= 0 else [] for p in parents]
        start = np.where(parents >= 0, old[parents], 0)
        assert all(lens[j] in (start[j], start[j] + grow[j]) for j in range(m))
        assert state[2] == (lens != start + grow).sum()
        missed += state[2]
        for j in range(m):
            for t in range(start[j], lens[j]):
                texts[j].append(int(rng.integers(1, 1 << 30)))
                pool[tables[j, t // page], t % page] = texts[j][-1]
        n = m
        for j in range(n):
            assert [int(pool[tables[j, t // page], t % page]) for t in range(lens[j])] == texts[j]
    assert missed
