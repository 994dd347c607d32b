"""Forks that run out of pages, against their definition: every value equal,
and every sequence's tokens still in its pages."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from decode_util import ints
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu


def _fork(tables, lens, refs, page, parents, grow, pools=()):
    host = [p.cpu().numpy().copy() for p in pools]
    ref = decode.fork(tables, lens, refs, page, parents, grow, host)
    got = i8.cache_fork(ints(tables), ints(lens), ints(refs), page, ints(parents), ints(grow), pools)
    torch.cuda.synchronize()
    for a, b, name in zip(got, ref, ("tables", "lens", "refs", "state")):
        assert np.array_equal(a.cpu().numpy(), b), (name, a.cpu().numpy(), b)
    for p, h in zip(pools, host):
        assert np.array_equal(p.cpu().numpy(), h)
    return ref


@pytest.mark.parametrize("seed", range(10))
def test_a_random_history_in_a_small_pool(seed):
    rng = np.random.default_rng(seed)
    page, M, P, n = 16, 3, int(rng.integers(1, 12)), 6
    tables, lens, refs = np.full((n, M), -1, np.int32), np.zeros(n, np.int32), np.zeros(P, np.int32)
    pool = torch.zeros((P, page, 4), dtype=torch.int32, device=DEV)
    texts, short = [[] for _ in range(n)], 0
    say(f"  launch: forks in a pool of {P} pages, seed {seed}")
    for _ in range(30):
        m = int(rng.integers(1, 10))
        parents, grow = rng.integers(-1, n, size=m), rng.integers(0, 9 if seed % 2 else 45, size=m)
        old = lens
        tables, lens, refs, state = _fork(tables, lens, refs, page, parents, grow, [pool])
        short += state[2]
        texts = [list(texts[p]) if p >= 0 else [] for p in parents]
        host = pool.cpu().numpy()
        for j in range(m):
            for t in range(old[parents[j]] if parents[j] >= 0 else 0, lens[j]):
                texts[j].append(int(rng.integers(1, 1 << 30)))
                host[tables[j, t // page], t % page] = texts[j][-1]
        pool.copy_(torch.from_numpy(host))
        n = m
        for j in range(n):
            assert [int(host[tables[j, t // page], t % page, 0]) for t in range(lens[j])] == texts[j]
    assert short


@pytest.mark.parametrize("pages", [0, 40000])
@pytest.mark.parametrize("n,free", [(30, 11), (1000, 700), (1024, 0), (1025, 1023), (3000, 1500), (3000, 2998), (3000, 2999), (3000, 5000)])
def test_one_page_of_many_sequences_with_few_pages_free(n, free, pages):
    """All sequences write on in page 0, and every 50th asks for more than there is room for: who keeps a page may come
    many sequences behind the one that found none. In one launch and in several (more than 1024 sequences or 32768 pages)."""
    tables, lens = np.zeros((n, 2), np.int32), np.full(n, 5, np.int32)
    tables[:, 1] = -1
    refs = np.zeros(max(pages, free + 1), np.int32)
    refs[0], refs[free + 1:] = n, 1
    pool = torch.arange(len(refs), device=DEV, dtype=torch.int32)[:, None].repeat(1, 4).contiguous()
    say(f"  launch: cache_fork, {n} sequences in one page, {free} free of {len(refs)}")
    for unable in (False, True):
        grow = np.ones(n, np.int64)
        if unable:
            grow[7::50] = 100
        _, sizes, counts, state = _fork(tables, lens, refs, 16, np.arange(n), grow, [pool.clone()])
        enough = free >= n - 1 if not unable else free >= n - (grow > 1).sum()
        assert sizes[-1] == (6 if enough else 5) and state[2] == (sizes == 5).sum()
        assert counts.sum() == n + len(refs) - free - 1


def test_pages_shared_by_pairs_at_the_edge_of_what_is_free():
    """2600 sequences, neighbours and far apart, share last pages by twos and threes; the free pages end between them."""
    rng = np.random.default_rng(3)
    n, page = 2600, 16
    tables = np.full((n, 3), -1, np.int32)
    tables[:, 0] = rng.permutation(np.concatenate([np.arange(1300) // 2, 650 + np.arange(1300) // 3]))
    used = int(tables[:, 0].max()) + 1
    lens = rng.integers(1, 16, size=used).astype(np.int32)[tables[:, 0]]
    for free in (0, 1, 500, 1299, 1300, 1301, 2000, 2599, 2600, 4000):
        refs = np.concatenate([np.bincount(tables[:, 0], minlength=used), np.zeros(free, int)]).astype(np.int32)
        grow = rng.integers(0, 20, size=n)
        say(f"  launch: cache_fork, pairs, {free} free")
        _fork(tables, lens, refs, page, np.arange(n), grow, [torch.rand((len(refs), 4), device=DEV)])
        _fork(tables, lens, refs, page, rng.integers(-1, n, size=1000), rng.integers(0, 40, size=1000), [])
