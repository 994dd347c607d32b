"""The definitions of the paged cache and of beam search on cases worked out by
hand, and what must hold after any sequence of forks (CPU)."""

import numpy as np
import pytest

from oracle import decode

I = np.int32   # noqa: E741


def test_fork_shares_copies_frees_and_allocates():
    # page 16; sequence 0 holds 20 tokens on pages 4, 2; sequence 1 16 tokens on page 0
    tables, lens = np.array([[4, 2, -1], [0, 7, 7]], I), np.array([20, 16], I)
    refs = np.array([1, 0, 1, 0, 1, 0, 0, 0], I)
    pool = np.arange(8.0).reshape(8, 1).copy()
    t, n, r, s = decode.fork(tables, lens, refs, 16, [0, 0, 1], [1, 13, 1], [pool])
    # the first of the two copies page 2 to page 1; the second keeps it and takes page 3 behind it; then page 5
    assert t.tolist() == [[4, 1, -1], [4, 2, 3], [0, 5, -1]] and n.tolist() == [21, 33, 17]
    assert r.tolist() == [1, 1, 1, 1, 2, 1, 0, 0] and s.tolist() == [2, 0, 0, 1]
    assert pool[:, 0].tolist() == [0, 2, 2, 3, 4, 5, 6, 7]
    # nobody goes on from sequence 0, slot 1 starts empty
    t, n, r, s = decode.fork(tables, lens, refs, 16, [1, -1], [0, 17])
    assert t.tolist() == [[0, -1, -1], [1, 2, -1]] and n.tolist() == [16, 17]
    assert r.tolist() == [1, 1, 1, 0, 0, 0, 0, 0] and s.tolist() == [5, 0, 0, 0]


def test_fork_without_room():
    tables, lens, refs = np.array([[0, -1], [1, -1], [2, 3]], I), np.array([16, 16, 32], I), np.array([1, 1, 1, 1, 0], I)
    t, n, r, s = decode.fork(tables, lens, refs, 16, None, [1, 1, 1])
    assert n.tolist() == [17, 16, 32] and t.tolist() == [[0, 4], [1, -1], [2, 3]]
    assert r.tolist() == [1, 1, 1, 1, 1] and s.tolist() == [0, 1, 2, 0]


def test_compact_moves_the_tail_into_the_gaps():
    refs, pool = np.array([0, 2, 0, 0, 1, 3], I), np.arange(6.0)[:, None].copy()
    t, r, moved, s = decode.compact(np.array([[1, 4, -1], [1, 5, 99]], I), refs, [pool])
    assert moved.tolist() == [-1, 1, -1, -1, 0, 2] and r.tolist() == [1, 2, 3, 0, 0, 0] and s.tolist() == [3, 2]
    assert t.tolist() == [[1, 0, -1], [1, 2, 99]] and pool[:3, 0].tolist() == [4, 1, 5]


def test_select_worked_example():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]]))
    s, p, t, h = decode.select(x, np.array([[0.0, np.log(0.5)]]), 4, np.array([[7], [8]]))
    assert np.allclose(np.exp(s), [[0.5, 0.4, 0.25, 0.25]])
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 2, 1, 2]] and h.tolist() == [[7, 0], [8, 2], [7, 1], [7, 2]]
    s, p, t, _ = decode.select(np.array([[np.nan, 1.0], [-np.inf, 0.0]]), np.array([[0.0, -1.0]]), 3)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[1, 0, 1]] and s[0, 0] == -1.0 and np.isneginf(s[0, 1:]).all()


def test_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(0)
    V = rng.normal(size=(3, 2, 16, 8))
    out, lse = decode.attention(np.ones((1, 32)), np.zeros_like(V), V, np.array([[2, 0, 1]], I), [37], 0.3)
    rows = np.concatenate([V[2], V[0], V[1][:, :5]], 1).mean(1)
    assert np.allclose(out.reshape(4, 8), rows[[0, 0, 1, 1]]) and np.allclose(lse, np.log(37))
    out, lse = decode.attention(np.ones((1, 32)), np.zeros_like(V), V, np.array([[9, 0, -1]], I), [40], 0.3)
    assert np.allclose(out.reshape(4, 8)[0], V[0, 0].mean(0)) and np.allclose(lse, np.log(16))
    out, lse = decode.attention(np.ones((2, 32)), V, V, np.array([[9], [0]], I), [16, 0], 0.3)
    assert not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("seed", range(20))
def test_counts_agree_and_no_written_page_is_shared(seed):
    rng = np.random.default_rng(seed)
    page, M, P, n = 16, 4, int(rng.integers(8, 60)), 5
    tables, lens, refs = np.full((n, M), -1, I), np.zeros(n, I), np.zeros(P, I)
    texts, pool = [[] for _ in range(n)], np.zeros((P, page), I)     # what each sequence holds, and the cache
    for _ in range(40):
        n2 = int(rng.integers(1, 8))
        parents, grow = rng.integers(-1, n, size=n2), rng.integers(0, 9, size=n2)
        old = lens
        tables, lens, refs, state = decode.fork(tables, lens, refs, page, parents, grow, [pool])
        texts = [list(texts[p]) if p >= 0 else [] for p in parents]
        if rng.random() < 0.3:
            tables, refs, _, _ = decode.compact(tables, refs, [pool])
        for j in range(n2):
            start = old[parents[j]] if parents[j] >= 0 else 0
            assert lens[j] in (start, start + grow[j])
            for t in range(start, lens[j]):
                texts[j].append(int(rng.integers(1, 1 << 30)))
                pool[tables[j, t // page], t % page] = texts[j][-1]
        n = n2
        counts = np.zeros(P, I)
        for j in range(n):
            used = -(-lens[j] // page)
            assert (tables[j, :used] >= 0).all() and (tables[j, used:] == -1).all()
            np.add.at(counts, tables[j, :used], 1)
            assert [int(pool[tables[j, t // page], t % page]) for t in range(lens[j])] == texts[j]
        assert np.array_equal(counts, refs) and state[0] == (refs <= 0).sum()
