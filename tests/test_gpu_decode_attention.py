"""Attention of new tokens over a paged cache against its definition in 64 bits.

Bounds: decode_util.attention_bounds, derived from the number of roundings, and
half a step of the output's type."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, randn, strided, wide
from decode_util import attention_bounds, ints, paged, pool
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _near_lse(got, ref, bound):
    g = wide(got)
    empty = np.isneginf(ref)
    assert np.array_equal(np.isneginf(g), empty)
    assert (np.abs(g - np.where(empty, 0, ref))[~empty] <= bound[~empty]).all(), np.abs(g - ref)[~empty].max()


def _check(q, K, V, tables, lens, scale=None, slopes=None, beams=1, **kw):
    d = K.shape[3]
    t = tables if isinstance(tables, torch.Tensor) else ints(tables)
    out, lse = i8.decode_attention(q, K, V, t, ints(lens), scale=scale, slopes=slopes, beams=beams, **kw)
    torch.cuda.synchronize()
    tables = t.cpu().numpy()
    scale = d ** -0.5 if scale is None else scale
    sl = None if slopes is None else wide(slopes)
    ro, rl = decode.attention(wide(q), wide(K), wide(V), tables, lens, scale, sl)
    bo, bl = attention_bounds(q, K, V, tables, lens, scale, sl, q.dtype)
    near(out, ro, bo, "out")
    _near_lse(lse, rl, bl)
    return out, lse


def _wider(tables, page, keys=1040):
    """The same tables with room for so many positions: beyond 1024 the work is split and joined."""
    out = np.full((len(tables), max(tables.shape[1], -(-keys // page))), -1, np.int32)
    out[:, :tables.shape[1]] = tables
    return out


CASES = [
    # heads, kv_heads, d, page, lengths
    (1, 1, 64, 16, [1]), (1, 1, 8, 16, [5, 0, 33]), (3, 3, 24, 48, [100, 1, 49]), (4, 4, 80, 16, [16, 17, 15, 0, 128, 129]),
    (4, 2, 96, 32, [31, 32, 33, 127, 300]), (12, 12, 64, 16, [131]), (8, 1, 128, 64, [63, 64, 65, 640]),
    (5, 5, 128, 16, [1, 2, 257, 500]), (16, 1, 128, 16, [129, 700]), (24, 1, 64, 16, [40, 513]), (34, 2, 128, 32, [77, 257]),
    (6, 3, 256, 16, [1, 130, 260]), (2, 1, 200, 16, [19, 255]), (2, 2, 136, 4096, [4097, 3]), (2, 1, 112, 1008, [1009, 1008]),
    (2, 2, 128, 16, [2500]), (1, 1, 64, 16, [9001, 3]), (7, 7, 40, 32, [64] * 9), (1, 1, 128, 128, list(range(0, 300, 23)))]


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", CASES, ids=[str(c[:4]) + str(len(c[4])) for c in CASES])
def test_against_the_definition(case, dtype, alibi):
    heads, kv, d, page, lens = case
    rng = np.random.default_rng(heads * 1000 + d + len(lens))
    tables, pages = paged(rng, lens, page)
    say(f"  launch: decode_attention {case[:4]}, {len(lens)} sequences, {dtype}, alibi {alibi}")
    K, V = (pool(rng, tables, lens, pages, kv, page, d, dtype) for _ in range(2))
    q = randn(rng, (len(lens), heads * d), dtype, 1.5)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device=DEV) if alibi else None
    _check(q, K, V, tables, lens, slopes=slopes)
    _check(q, K, V, _wider(tables, page), lens, slopes=slopes)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_strides_and_what_lies_around(dtype):
    """Queries and outputs as parts of wider rows, pages apart, a table with its own stride and more columns than are used;
    rows and columns beyond are left as they were."""
    rng = np.random.default_rng(5)
    lens, page, heads, kv, d = [20, 0, 97, 64], 16, 6, 2, 64
    tables, pages = paged(rng, lens, page, width=11)
    K, V = (pool(rng, tables, lens, pages, kv, page, d, dtype, gap) for gap in (0, 40))
    q = strided(randn(rng, (4, heads * d), dtype), 2 * kv * d, 8)
    table = torch.full((4, 17), 1 << 30, dtype=torch.int32, device=DEV)
    table[:, :11] = ints(tables)
    out = strided(torch.zeros((4, heads * d), dtype=dtype, device=DEV), 24, 16)
    lse = torch.zeros((4, heads), device=DEV)
    say("  launch: decode_attention, strided")
    got, got_lse = _check(q, K, V, table[:, :11], lens, out=out, lse=lse)
    assert got.data_ptr() == out.data_ptr() and got_lse.data_ptr() == lse.data_ptr()
    store = torch.as_strided(out, (4, heads * d + 24), (heads * d + 24, 1))
    assert torch.isnan(store[:, heads * d:]).all()


def test_lengths_and_pages_that_do_not_exist():
    """Negative lengths are 0, lengths beyond the table end with it, page numbers outside the pool hold nothing."""
    rng = np.random.default_rng(6)
    page, heads, d = 16, 4, 64
    lens = [80, 80, 80, -5, 10 ** 9, 2 ** 31 - 1, -2 ** 31, 80, 33]
    full = [80] * 9
    tables, pages = paged(rng, full, page)
    K, V = (pool(rng, tables, full, pages, heads, page, d, F16) for _ in range(2))
    tables[0, 1], tables[1, 4], tables[2, :] = -1, pages, [pages, -1, 2 ** 31 - 1, -2 ** 31, pages + 7]
    tables[7, 0], tables[7, 3], tables[8, 2] = 2 ** 31 - 1, -2 ** 31, -7
    q = randn(rng, (9, heads * d), F16)
    say("  launch: decode_attention, lengths and pages that do not exist")
    _check(q, K, V, tables, lens, slopes=torch.full((heads,), 0.1, device=DEV))
    _check(q, K, V, _wider(tables, page), lens, slopes=torch.full((heads,), 0.1, device=DEV))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_scores_and_far_biases(dtype):
    """Scores far apart (one key takes all the weight), all equal, and a bias that leaves the last keys only."""
    rng = np.random.default_rng(7)
    lens, page, d = [300, 300, 300], 16, 64
    tables, pages = paged(rng, lens, page)
    K, V = pool(rng, tables, lens, pages, 2, page, d, dtype, std=30.0), pool(rng, tables, lens, pages, 2, page, d, dtype)
    q = randn(rng, (3, 4 * d), dtype, 20.0)
    q[1] = 0
    say(f"  launch: decode_attention, large scores, {dtype}")
    _check(q, K, V, tables, lens)
    _check(q, K, V, tables, lens, scale=-0.01)
    _check(q, K, V, tables, lens, scale=0.0, slopes=torch.tensor([50.0, -50.0, 3.0, 0.0], device=DEV))
    _check(q, K, V, tables, lens, scale=1e-4, slopes=torch.tensor([1e-6, 1.0, -1.0, 1e4], device=DEV))
    tables = _wider(tables, page)
    _check(q, K, V, tables, lens)
    _check(q, K, V, tables, lens, scale=0.0, slopes=torch.tensor([50.0, -50.0, 3.0, 0.0], device=DEV))


def test_small_weights_are_not_lost():
    """One key far above thousands that share the rest of the weight: e^-11 each, 4000 of them."""
    rng = np.random.default_rng(8)
    for dtype in (F16, BF16):
        n, page, d = 4001, 32, 64
        tables, pages = paged(rng, [n], page)
        K, V = pool(rng, tables, [n], pages, 1, page, d, dtype, std=0.0), pool(rng, tables, [n], pages, 1, page, d, dtype, std=0.0)
        V += 1
        at = int(tables[0, 3])
        K[at, 0, 5, 0], V[at, 0, 5] = 11.0, -1.0
        q = torch.zeros((1, d), dtype=dtype, device=DEV)
        q[0, 0] = 1.0
        say(f"  launch: decode_attention, small weights, {dtype}")
        _check(q, K, V, tables, [n], scale=1.0)


def test_values_near_the_ends_of_the_types():
    """bf16 values near fp32's end and near its smallest numbers, fp16's largest: nothing overflows or vanishes on the way."""
    rng = np.random.default_rng(19)
    lens, page, d = [3, 2, 700], 16, 64
    tables, pages = paged(rng, lens, page)
    for dtype, std in ((BF16, 2.0e37), (BF16, 1e-30), (F16, 9000.0), (F16, 1e-5)):
        say(f"  launch: decode_attention, values of {std}, {dtype}")
        n = lens if std < 1e30 else [3, 2, 5]             # the sum of a few such values is still a number of fp32
        K, V = pool(rng, tables, n, pages, 2, page, d, dtype), pool(rng, tables, n, pages, 2, page, d, dtype, std=std)
        q = randn(rng, (3, 2 * d), dtype)
        _check(q, K, V, tables, n)
        _check(q, K, V, _wider(tables, page), n)


def test_values_that_are_not_finite():
    """A NaN or infinity among a sequence's tokens reaches the heads that read it alone, as the definition says; behind the
    last token (the pools are NaN there) and in other sequences it reaches nothing."""
    rng = np.random.default_rng(9)
    lens, page, kv, d = [90, 90, 90, 90], 16, 3, 64
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, kv, page, d, F16) for _ in range(2))
    q = randn(rng, (4, 2 * kv * d), F16)
    K[int(tables[0, 2]), 1, 3, 7] = float("nan")
    V[int(tables[1, 5]), 2, 9, 11] = float("inf")
    V[int(tables[2, 0]), 0, 0, 0] = float("nan")
    K[int(tables[3, 1]), 0, 4, :] = 65504.0
    q[3, :2 * d] = 65504.0
    for table in (tables, _wider(tables, page)):
        _not_finite(q, K, V, tables, table, lens, d)


def _not_finite(q, K, V, tables, table, lens, d):
    say("  launch: decode_attention, values that are not finite")
    out, lse = i8.decode_attention(q, K, V, ints(table), ints(lens))
    torch.cuda.synchronize()
    o, s = wide(out).reshape(4, 6, d), wide(lse)
    assert np.isnan(o[0, 2:4]).all() and np.isnan(s[0, 2:4]).all()
    assert np.isposinf(o[1, 4:6, 11]).all() and np.isnan(o[2, :2, 0]).all()
    good = np.ones((4, 6, d), bool)
    good[0, 2:4], good[1, 4:6, 11], good[2, :2, 0] = False, False, False
    assert np.isfinite(o[good]).all() and np.isfinite(np.delete(s, 0, 0)).all()
    # one key's score of 2^39 or so takes all the weight
    assert np.array_equal(o[3, 0], wide(V[int(tables[3, 1]), 0, 4]))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_pools_beyond_32_bit_offsets(dtype):
    """Pages behind the 4th GiB of a pool, in elements and in bytes."""
    rng = np.random.default_rng(10)
    heads, page, d = 64, 64, 128
    pages = 2 ** 32 // (heads * page * d) + 9         # 2^32 elements and some
    K, V = (torch.empty((pages, heads, page, d), dtype=dtype, device=DEV) for _ in range(2))
    lens, tables = [130, 70], np.array([[pages - 1, 3, pages - 2], [pages // 2 + 1, 0, -1]], np.int32)
    for p in (K, V):
        for id in tables[tables >= 0]:
            p[int(id)] = randn(rng, (heads, page, d), dtype)
    q = randn(rng, (2, heads * d), dtype)
    say("  launch: decode_attention over 2 x 8.6 GB")
    out, lse = i8.decode_attention(q, K, V, ints(tables), ints(lens))
    ids = [int(i) for i in np.unique(tables[tables >= 0])]
    small = np.array([[ids.index(i) if i >= 0 else -1 for i in row] for row in tables], np.int32)
    few = slice(0, 3)                                  # three heads of each, in 64 bits
    K, V = K[ids][:, few].contiguous(), V[ids][:, few].contiguous()
    torch.cuda.synchronize()
    ro, rl = decode.attention(wide(q)[:, :3 * d], wide(K), wide(V), small, lens, d ** -0.5)
    bo, bl = attention_bounds(q[:, :3 * d], K, V, small, lens, d ** -0.5, None, dtype)
    near(out[:, :3 * d], ro, bo, "out")
    _near_lse(lse[:, :3], rl, bl)


def _beam_tables(rng, groups, beams, page, shared, own):
    """Groups of sequences that share `shared` pages and have `own` tokens (each their own number) after them."""
    lens, rows, free = [], [], list(rng.permutation(groups * (shared + beams * (max(own) // page + 2)) + 5))
    pages = len(free)
    for _ in range(groups):
        common = [free.pop() for _ in range(shared)]
        for b in range(beams):
            n = shared * page + own[b % len(own)]
            lens.append(n)
            rows.append(common + [free.pop() for _ in range(-(-n // page) - shared)])
    width = max(map(len, rows))
    return lens, np.array([r + [-1] * (width - len(r)) for r in rows], np.int32), pages


@pytest.mark.parametrize("heads,kv,d,page,beams,shared,own", [
    (4, 4, 128, 16, 4, 20, [5, 45, 16, 0]), (8, 8, 64, 32, 2, 3, [1, 100]), (6, 2, 80, 16, 3, 0, [7, 90, 33]),
    (8, 1, 128, 16, 5, 33, [3]), (16, 1, 64, 16, 4, 9, [20, 21]), (2, 2, 128, 16, 16, 17, [1, 2, 3]), (2, 1, 256, 16, 7, 6, [0, 9]),
    (1, 1, 128, 64, 33, 4, [10, 70, 1]), (3, 1, 64, 16, 64, 8, [3, 18])])
def test_beams_that_share_pages(heads, kv, d, page, beams, shared, own):
    rng = np.random.default_rng(heads + beams)
    lens, tables, pages = _beam_tables(rng, 2, beams, page, shared, own)
    K, V = (pool(rng, tables, lens, pages, kv, page, d, F16) for _ in range(2))
    q = randn(rng, (2 * beams, heads * d), F16)
    slopes = torch.tensor([0.5 / (h + 1) for h in range(heads)], device=DEV)
    tables = _wider(tables, page, 528)                # beyond what beams take whole
    say(f"  launch: decode_attention, {beams} beams, {heads} heads of {kv}, shared {shared}")
    _check(q, K, V, tables, lens, slopes=slopes, beams=beams)
    # pages that only some share, at other places of their rows, and lengths that differ over shared pages
    n = len(lens)
    tables[1], lens[1] = tables[0], max(1, lens[0] - 3)
    if n > 4:
        tables[3, :1], lens[3] = tables[n - 1, :1], min(lens[3], page)
        lens[2] = 0
    # a cache of NaN-free pages: other sequences' slots may lie behind a shorter one's last token
    K, V = torch.nan_to_num(K, nan=3.0), torch.nan_to_num(V, nan=7.0)
    _check(q, K, V, tables, lens, slopes=slopes, beams=beams)


def test_same_result_every_time_and_on_another_stream():
    rng = np.random.default_rng(12)
    lens, page, kv, d = [1000, 3, 517, 64], 16, 4, 128
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, kv, page, d, F16) for _ in range(2))
    q, t, n = randn(rng, (4, 8 * d), F16), ints(_wider(tables, page)), ints(lens)
    say("  launch: decode_attention, repeated")
    first = i8.decode_attention(q, K, V, t, n)
    ws = torch.empty(i8.decode_attention_workspace(4, 8, kv, d), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        again = i8.decode_attention(q, K, V, t, n, workspace=ws)
        with torch.cuda.stream(side):
            other = i8.decode_attention(q, K, V, t, n)
        torch.cuda.synchronize()
        ws.random_(0, 255)
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, other))


def test_captured_and_replayed():
    """Two graphs over one workspace, replayed in turn with new lengths, tables and queries."""
    rng = np.random.default_rng(13)
    page, kv, d, n = 16, 2, 64, 5
    tables, pages = paged(rng, [200] * n, page)
    K, V = (pool(rng, tables, [200] * n, pages, kv, page, d, BF16) for _ in range(2))
    q, t, lens = randn(rng, (n, 4 * d), BF16), ints(_wider(tables, page)), ints([1] * n)
    ws = torch.empty(i8.decode_attention_workspace(n, 4, kv, d), dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(q), torch.empty((n, 4), device=DEV)) for _ in range(2)]
    say("  launch: decode_attention, captured")
    graphs = []
    for (out, lse), beams in zip(outs, (1, 5)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            i8.decode_attention(q, K, V, t, lens, out=out, lse=lse, beams=beams, workspace=ws)
        graphs.append(g)
    for k in range(5):
        q.copy_(randn(rng, tuple(q.shape), BF16))
        lens.copy_(ints(rng.integers(0, 201, size=n)))
        if k == 3:
            t[0] = t[1]
        for g, (out, lse), beams in zip(graphs, outs, (1, 5)):
            g.replay()
            eager = i8.decode_attention(q, K, V, t, lens, beams=beams)
            torch.cuda.synchronize()
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_many_sequences():
    """More sequences than any block walks through at once: short ones, their lengths 0 to 17."""
    rng = np.random.default_rng(14)
    n, page, d = 5000, 16, 64
    lens = rng.integers(0, 18, size=n)
    tables, pages = paged(rng, lens, page)
    K, V = (torch.from_numpy(rng.normal(size=(pages, 1, page, d)).astype(np.float32)).to(DEV).half() for _ in range(2))
    q = randn(rng, (n, d), F16)
    say("  launch: decode_attention, 5000 sequences")
    _check(q, K, V, tables, lens)
    tables = _wider(tables, page)
    _check(q, K, V, tables, lens)
    _check(q, K, V, tables, lens, beams=10)


@pytest.mark.parametrize("heads,kv,d,keys", [(3, 1, 64, 133000), (1, 1, 40, 131072), (6, 1, 128, 70000)])
def test_one_long_sequence(heads, kv, d, keys):
    """A result that is joined of more parts than any other test's: up to 1024 of them."""
    rng = np.random.default_rng(heads)
    lens = [keys, 5]
    tables, pages = paged(rng, lens, 64)
    K, V = (pool(rng, tables, lens, pages, kv, 64, d, F16) for _ in range(2))
    q = randn(rng, (2, heads * d), F16, 1.5)
    say(f"  launch: decode_attention, {keys} tokens, {heads} heads of {d}")
    _check(q, K, V, tables, lens)
    _check(q, K, V, tables, lens, slopes=torch.full((heads,), 2.0 ** -12, device=DEV))


def test_no_sequences_and_refusals():
    K = torch.zeros((4, 2, 16, 64), dtype=F16, device=DEV)
    q = torch.zeros((2, 256), dtype=F16, device=DEV)
    t, n = ints([[0, 1], [2, 3]]), ints([20, 5])
    out, lse = i8.decode_attention(q[:0], K, K, t[:0], n[:0])
    assert out.shape == (0, 256) and lse.shape == (0, 4)
    for kw in (dict(q=q.float()), dict(q=q.bfloat16()), dict(q=q.cpu()), dict(K=K[:, :1]), dict(V=K.bfloat16()),
               dict(K=K.transpose(1, 2)), dict(t=t.long()), dict(t=t[:1]), dict(n=n[:1]), dict(n=n.long()), dict(q=q[:, :100]),
               dict(slopes=torch.zeros(3, device=DEV)), dict(workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
               dict(lse=torch.zeros((2, 2), device=DEV)), dict(out=torch.zeros((2, 128), dtype=F16, device=DEV))):
        a = dict(q=q, K=K, V=K, t=t, n=n)
        extra = {k: v for k, v in kw.items() if k not in a}
        a.update({k: v for k, v in kw.items() if k in a})
        with pytest.raises((ValueError, TypeError, i8.I8MMError)):
            i8.decode_attention(a["q"], a["K"], a["V"], a["t"], a["n"], **extra)
    for kw in (dict(beams=3), dict(beams=0), dict(scale=float("nan")), dict(out=q)):
        with pytest.raises(i8.I8MMError):
            i8.decode_attention(q, K, K, t, n, **kw)
    with pytest.raises(i8.I8MMError):
        i8.decode_attention(q, K.reshape(8, 2, 8, 64), K.reshape(8, 2, 8, 64), t, n)
