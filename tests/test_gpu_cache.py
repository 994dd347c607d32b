"""The paged cache's bookkeeping and copies against their definitions: every
value equal."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import randn, strided
from decode_util import ints, paged
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _bits(t):
    return t.view(torch.int16).cpu().numpy()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,d,page,s", [(1, 8, 16, 1), (12, 64, 16, 5), (96, 128, 16, 64), (3, 80, 48, 300), (2, 256, 4096, 33),
                                            (32, 128, 32, 1000), (5, 24, 16, 77), (65, 200, 16, 9)])
def test_append(heads, d, page, s, dtype):
    rng = np.random.default_rng(heads + d)
    n, room = 6, max(2 * page, s)
    tables, pages = paged(rng, [room] * n, page)
    seq, pos = np.arange(s) % n, np.arange(s) // n + rng.integers(0, page, size=n)[np.arange(s) % n]
    # rows that are left out: sequences, positions and pages that do not exist
    for k, (a, b) in enumerate([(-1, 0), (n, 0), (2 ** 31 - 1, 3), (0, -1), (1, tables.shape[1] * page), (2, 2 ** 31 - 1),
                                (-2 ** 31, -2 ** 31)]):
        if s > 20:
            seq[3 * k], pos[3 * k] = a, b
    tables[3, 0], tables[4, 0] = -1, pages
    wide_row = strided(randn(rng, (s, 2 * heads * d), dtype), 16, 8)
    K, V = wide_row[:, :heads * d], wide_row[:, heads * d:]
    store = randn(rng, (2, pages, heads * page * d + 8), dtype)
    Kp, Vp = (p[:, :heads * page * d].view(pages, heads, page, d) for p in store)
    ref = _bits(store).copy()
    Kr, Vr = (p[:, :heads * page * d].reshape(pages, heads, page, d) for p in ref)     # copies, as the gap splits them
    decode.append(_bits(K.contiguous()), _bits(V.contiguous()), Kr, Vr, tables, pos, seq)
    say(f"  launch: cache_append {heads} x {d}, page {page}, {s} rows, {dtype}")
    i8.cache_append(K, V, Kp, Vp, ints(tables), ints(pos), ints(seq))
    torch.cuda.synchronize()
    assert np.array_equal(_bits(Kp.contiguous()), Kr) and np.array_equal(_bits(Vp.contiguous()), Vr)
    assert np.array_equal(_bits(store)[:, :, heads * page * d:], ref[:, :, heads * page * d:])
    if s <= n:                                      # one row a sequence: seq left out
        before = _bits(Kp.contiguous()).copy()
        i8.cache_append(V, K, Kp, Vp, ints(tables), ints(pos))
        torch.cuda.synchronize()
        decode.append(_bits(V.contiguous()), _bits(K.contiguous()), before, Vr, tables, pos)
        assert np.array_equal(_bits(Kp.contiguous()), before)


def test_append_rows_of_one_slot_and_far_pages():
    """Two rows for one slot: each 16 bytes are one of theirs. A page beyond 2^32 bytes."""
    heads, d, page = 32, 128, 64
    pages = 2 ** 32 // (heads * page * d) + 3
    Kp = torch.empty((pages, heads, page, d), dtype=F16, device=DEV)
    K = torch.stack([torch.full((heads * d,), v, dtype=F16, device=DEV) for v in (1.0, 2.0)])
    say("  launch: cache_append, one slot twice, 8.6 GB pool")
    i8.cache_append(K, K, Kp, Kp, ints([[pages - 1, 0]]), ints([5, 5]), ints([0, 0]))
    got = Kp[pages - 1, :, 5].reshape(-1, 8)
    torch.cuda.synchronize()
    assert ((got == 1).all(1) | (got == 2).all(1)).all()


def _run_fork(tables, lens, refs, page, parents, grow, pools, **kw):
    host = [p.cpu().numpy().copy() for p in pools]
    ref = decode.fork(tables, lens, refs, page, parents, grow, host)
    got = i8.cache_fork(ints(tables), ints(lens), ints(refs), page, None if parents is None else ints(parents),
                        None if grow is None else ints(grow), pools, **kw)
    torch.cuda.synchronize()
    for a, b, name in zip(got, ref, ("tables", "lens", "refs", "state")):
        assert np.array_equal(a.cpu().numpy(), b), (name, a.cpu().numpy(), b)
    for p, h in zip(pools, host):
        assert np.array_equal(p.cpu().numpy(), h)
    return ref


@pytest.mark.parametrize("seed", range(12))
def test_a_random_history_of_forks_and_compactions(seed):
    rng = np.random.default_rng(seed)
    page, M, P, n = int(rng.choice([16, 32])), int(rng.integers(1, 6)), int(rng.integers(1, 90)), int(rng.integers(0, 7))
    tables, lens, refs = np.full((n, M), -1, np.int32), np.zeros(n, np.int32), np.zeros(P, np.int32)
    pools = [torch.randint(0, 127, (P, 3, 16), device=DEV, dtype=torch.int8), torch.rand((P, 4), device=DEV),
             torch.rand((P, 40), device=DEV)[:, 4:12]]
    say(f"  launch: forks and compactions, seed {seed}")
    for step in range(14):
        m = int(rng.integers(0, 12))
        parents = None if m == n and step % 3 == 0 else rng.integers(-2, n + 2, size=m)
        grow = None if step % 5 == 4 and parents is not None else rng.integers(-1, 2 * page, size=m) * (rng.random(m) < 0.7)
        tables, lens, refs, _ = _run_fork(tables, lens, refs, page, parents, grow, pools)
        n = m
        if step % 4 == 3:
            host = [p.cpu().numpy().copy() for p in pools]
            ref = decode.compact(tables, refs, host)
            got = i8.cache_compact(ints(tables), ints(refs), pools)
            torch.cuda.synchronize()
            for a, b in zip(got, ref):
                assert np.array_equal(a.cpu().numpy(), b)
            for p, h in zip(pools, host):
                assert np.array_equal(p.cpu().numpy(), h)
            tables, refs = ref[0], ref[1]


def test_fork_with_counts_and_pages_that_do_not_agree():
    """Counts a caller added to, counts below zero, page numbers outside the pool, lengths out of range."""
    tables = np.array([[0, 9, 2, -1], [3, -7, 2 ** 31 - 1, 4], [5, 6, -2 ** 31, 1], [7, 7, 7, 7]], np.int32)
    lens, refs = np.array([40, 10 ** 9, -3, 63]), np.array([2, 1, 3, -4, 1, 0, 0, 1], np.int32)
    pools = [torch.rand((8, 16), device=DEV)]
    say("  launch: cache_fork, counts that do not agree")
    for parents, grow in (([0, 1, 2, 3], [1, 1, 1, 1]), ([3, 3, 3, 0, 0], [1, 0, 1, 9, 2 ** 31 - 1]), ([2 ** 31 - 1, -2 ** 31], [5, 0]),
                          (None, None), ([1, 1], None), (None, [0, 3, 40, -2 ** 31])):
        _run_fork(tables, lens, refs, 16, parents, grow, pools)


def _many(rng, requests, beams, page, shared, mine, spare):
    ids = list(rng.permutation(requests * (shared + beams * mine) + spare))
    P, refs, rows = len(ids), np.zeros(len(ids), np.int32), []
    for _ in range(requests):
        common = [ids.pop() for _ in range(shared)]
        rows += [common + [ids.pop() for _ in range(mine)] for _ in range(beams)]
    tables = np.array([r + [-1, -1] for r in rows], np.int32)
    np.add.at(refs, tables[tables >= 0], 1)
    return tables, refs, P


@pytest.mark.parametrize("requests,beams,shared,mine,spare", [(300, 8, 11, 2, 20000), (1, 64, 500, 1, 3), (2500, 1, 0, 30, 100),
                                                              (40, 4, 100, 3, 300), (1200, 2, 1, 1, 100000),
                                                              (128, 8, 20, 2, 28160), (128, 8, 20, 2, 28161), (205, 5, 9, 2, 50)])
def test_fork_and_compact_of_many_sequences(requests, beams, shared, mine, spare):
    rng = np.random.default_rng(requests)
    page = 16
    tables, refs, P = _many(rng, requests, beams, page, shared, mine, spare)
    n = requests * beams
    lens = (shared + mine) * page - rng.integers(0, page, size=requests).repeat(beams)
    parents = np.arange(n) // beams * beams + rng.integers(0, beams, size=n)
    grow = rng.integers(0, 20, size=n)
    pools = [torch.randint(-2 ** 31, 2 ** 31 - 1, (P, 12), device=DEV, dtype=torch.int32)]
    say(f"  launch: cache_fork of {n} sequences, {P} pages")
    tables, lens, refs, state = _run_fork(tables, lens, refs, page, parents, grow, pools)
    assert state[3] > 0 or beams == 1
    host = [p.cpu().numpy().copy() for p in pools]
    ref = decode.compact(tables, refs, host)
    t = ints(tables)
    got = i8.cache_compact(t, ints(refs), pools, tables_out=t)           # in place
    torch.cuda.synchronize()
    assert got[0].data_ptr() == t.data_ptr()
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(pools[0].cpu().numpy(), host[0])


@pytest.mark.parametrize("P,share", [(1, 0.0), (1, 1.0), (4096, 0.5), (4097, 0.9), (20000, 0.0), (20000, 1.0), (70001, 0.3)])
def test_compact_pools_of_any_size(P, share):
    rng = np.random.default_rng(P)
    refs = (rng.random(P) < share) * rng.integers(1, 4, size=P) - (rng.random(P) < 0.1) * (rng.random(P) < 1 - share)
    refs = refs.astype(np.int32)
    tables = rng.integers(-1, P + 1, size=(7, 13)).astype(np.int32)
    pools = [torch.rand((P, 8), device=DEV)]
    host = [pools[0].cpu().numpy().copy()]
    ref = decode.compact(tables, refs, host)
    say(f"  launch: cache_compact of {P} pages, {share} in use")
    got = i8.cache_compact(ints(tables), ints(refs), pools)
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(pools[0].cpu().numpy(), host[0])


def test_many_pools_of_different_sizes():
    """More pools than one launch takes; pages of 16 bytes to several pieces of a block, with gaps."""
    rng = np.random.default_rng(4)
    P, sizes = 10, [int(rng.choice([16, 48, 4096, 16384, 16400, 70000 // 16 * 16])) for _ in range(150)]
    pools = [torch.randint(0, 255, (P, b + 16), device=DEV, dtype=torch.uint8)[:, :b] for b in sizes]
    tables, refs = np.array([[3, 8, -1], [3, 9, -1], [0, 5, 7]], np.int32), np.zeros(P, np.int32)
    np.add.at(refs, tables[tables >= 0], 1)
    say("  launch: cache_fork and cache_compact over 150 pools")
    tables, lens, refs, state = _run_fork(tables, np.array([20, 30, 45]), refs, 16, [0, 0, 0, 2], [1, 1, 1, 1], pools)
    assert state[3] == 2
    host = [p.cpu().numpy().copy() for p in pools]
    ref = decode.compact(tables, refs, host)
    i8.cache_compact(ints(tables), ints(refs), pools)
    torch.cuda.synchronize()
    for p, h in zip(pools, host):
        assert np.array_equal(p.cpu().numpy(), h)
    assert ref[3][1] > 0


def test_pages_beyond_32_bit_offsets():
    P, width = 5, 2 ** 30 + 16                          # pages a GiB apart
    store = torch.empty((P, width), dtype=torch.uint8, device=DEV)
    view = store[:, :4096]
    view.random_(0, 255)
    host = [view.cpu().numpy().copy()]
    ref = decode.compact(np.array([[4, 3]], np.int32), np.array([0, 0, 0, 1, 1], np.int32), host)
    say("  launch: cache_compact, pages a GiB apart")
    got = i8.cache_compact(ints([[4, 3]]), ints([0, 0, 0, 1, 1]), [view])
    torch.cuda.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), ref[0]) and np.array_equal(view.cpu().numpy(), host[0])


def test_fork_captured_and_replayed():
    """A captured step over outputs that are its next inputs' copies, one workspace for both calls."""
    rng = np.random.default_rng(3)
    tables, refs, P = _many(rng, 6, 4, 16, 3, 1, 40)
    lens = np.full(24, 60)
    t, n, r = ints(tables), ints(lens), ints(refs)
    parents, grow = ints(np.zeros(24)), ints(np.zeros(24))
    pools = [torch.rand((P, 64), device=DEV)]
    ws = torch.empty(max(i8.cache_fork_workspace(24, 24, P), i8.cache_compact_workspace(P)), dtype=torch.uint8, device=DEV)
    outs = dict(tables_out=torch.empty_like(t), lens_out=torch.empty_like(n), refs_out=torch.empty_like(r))
    packed = dict(tables_out=torch.empty_like(t), refs_out=torch.empty_like(r))
    say("  launch: cache_fork and cache_compact, captured")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, _, _, state = i8.cache_fork(t, n, r, 16, parents, grow, pools, workspace=ws, **outs)
        _, _, moved, _ = i8.cache_compact(outs["tables_out"], outs["refs_out"], pools, workspace=ws, **packed)
    for _ in range(6):
        par, gr = np.arange(24) // 4 * 4 + rng.integers(0, 4, size=24), rng.integers(0, 4, size=24)
        parents.copy_(ints(par))
        grow.copy_(ints(gr))
        host = [pools[0].cpu().numpy().copy()]
        a = decode.fork(t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy(), 16, par, gr, host)
        b = decode.compact(a[0], a[2], host)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(packed["tables_out"].cpu().numpy(), b[0]) and np.array_equal(moved.cpu().numpy(), b[2])
        assert np.array_equal(state.cpu().numpy(), a[3]) and np.array_equal(pools[0].cpu().numpy(), host[0])
        t.copy_(packed["tables_out"])
        n.copy_(outs["lens_out"])
        r.copy_(packed["refs_out"])


def test_refusals():
    t, n, r, pool = ints([[0, 1], [2, -1]]), ints([20, 5]), ints([1, 1, 1, 0]), torch.zeros((4, 4), device=DEV)
    for kw in (dict(parents=ints([0]), grow=ints([1, 1])), dict(parents=ints([0, 1]).long()), dict(pools=[pool[:3]]),
               dict(pools=[torch.zeros((4, 4, 4), device=DEV).transpose(1, 2)]), dict(pools=[pool.cpu()]),
               dict(pools=[torch.zeros((4, 3), device=DEV)]), dict(tables_out=t), dict(lens_out=n), dict(refs_out=r),
               dict(tables_out=ints([[0]])), dict(workspace=torch.zeros(4, dtype=torch.uint8, device=DEV))):
        with pytest.raises((ValueError, i8.I8MMError)):
            i8.cache_fork(t, n, r, 16, **kw)
    with pytest.raises(i8.I8MMError):
        i8.cache_fork(t, n, r, 8)
    with pytest.raises(i8.I8MMError):
        i8.cache_compact(t, r, refs_out=r)
    with pytest.raises(ValueError):
        i8.cache_compact(t.long(), r)
    K, x = torch.zeros((4, 2, 16, 64), dtype=F16, device=DEV), torch.zeros((2, 128), dtype=F16, device=DEV)
    for a in ((x, x[:1], K, K, t, n), (x.float(), x, K, K, t, n), (x, x, K, K[:2], t, n), (x, x, K, K, t, n[:1]),
              (x[:, :64], x, K, K, t, n), (x, x, K, K, t, n.long()), (x, x, K.transpose(2, 3), K, t, n)):
        with pytest.raises(ValueError):
            i8.cache_append(*a)
    i8.cache_append(x[:0], x[:0], K, K, t, n[:0])
