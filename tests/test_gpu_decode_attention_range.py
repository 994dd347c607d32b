"""Attention where fp32 has no room for a sum or a score, though the result is a number: against the definition in 64 bits.

A head that leaves fp32's range is computed in 64 bits, the others in fp32: decode_util.attention_bounds holds for both."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, randn, wide
from decode_util import attention_bounds, ints, paged, pool
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def _wider(tables, page, keys=1040):
    """The same tables with room for so many positions: beyond 1024 the work is split and joined."""
    out = np.full((len(tables), max(tables.shape[1], -(-keys // page))), -1, np.int32)
    out[:, :tables.shape[1]] = tables
    return out


def _check(q, K, V, tables, lens, scale=None, slopes=None, beams=1):
    d = K.shape[3]
    scale = d ** -0.5 if scale is None else scale
    sl = None if slopes is None else wide(slopes)
    ro, rl = decode.attention(wide(q), wide(K), wide(V), tables, lens, float(np.float32(scale)), sl)
    bo, bl = attention_bounds(q, K, V, tables, lens, scale, sl, q.dtype)
    for t in (tables, _wider(tables, K.shape[2])):
        out, lse = i8.decode_attention(q, K, V, ints(t), ints(lens), scale=scale, slopes=slopes, beams=beams)
        torch.cuda.synchronize()
        near(out, ro, bo, "out")
        some = np.isfinite(rl)
        assert np.array_equal(wide(lse)[~some], rl[~some], equal_nan=True)
        off = np.abs(wide(lse) - np.where(some, rl, 0))[some]
        assert (off <= bl[some]).all(), off.max()
    return ro


@pytest.mark.parametrize("dtype,value", [(BF16, 1e38), (BF16, 3.3e38), (F16, 65504.0)])
@pytest.mark.parametrize("heads,kv,d,page", [(1, 1, 64, 16), (4, 2, 128, 32), (16, 1, 80, 16), (18, 1, 128, 16), (2, 2, 256, 64), (3, 1, 8, 16)])
def test_sums_of_large_values(heads, kv, d, page, dtype, value):
    """Equal values, whose mean is their value and whose sum is far beyond fp32 (and, in fp16, whose weighted mean must not
    be rounded past the largest number); the same with signs, and in some heads and sequences alone."""
    rng = np.random.default_rng(heads)
    lens = [4, 1, 300, 700, 0, 2100]
    tables, pages = paged(rng, lens, page)
    K, V = pool(rng, tables, lens, pages, kv, page, d, dtype), pool(rng, tables, lens, pages, kv, page, d, dtype, std=0.0) + value
    say(f"  launch: decode_attention, values of {value}, {heads} heads on {kv}, {d}")
    q = randn(rng, (len(lens), heads * d), dtype)
    ref = _check(torch.zeros_like(q), K, V, tables, lens)
    assert np.allclose(np.delete(ref, 4, 0), float(torch.tensor(value, dtype=dtype)), rtol=1e-9)
    _check(q, K, V, tables, lens)
    V[:, 0] *= torch.tensor(np.where(rng.random((pages, page, 1)) < 0.3, -1.0, 1.0), device=DEV).to(dtype)
    _check(q, K, V, tables, lens)
    for i in (0, 3):                                  # ordinary numbers but in two sequences
        V[ints(tables[i][tables[i] >= 0]).long()] /= 2.0 ** 100 if dtype == BF16 else 2.0 ** 12
    _check(q, K, V, tables, lens)


@pytest.mark.parametrize("beams", [1, 4])
def test_some_of_many_heads_with_large_values(beams):
    """Blocks that write several heads each, of which some are beyond fp32."""
    rng = np.random.default_rng(beams)
    n, heads, d, page = 400, 6, 64, 16
    lens = list(rng.integers(0, 200, size=n))
    tables, pages = paged(rng, lens, page)
    if beams > 1:                                     # the first pages of a group are the first one's
        for i in range(n):
            k = min(lens[i], lens[i - i % beams]) // page
            tables[i, :k] = tables[i - i % beams, :k]
    K, V = (torch.nan_to_num(pool(rng, tables, lens, pages, heads, page, d, BF16)) for _ in range(2))
    far = torch.as_tensor(rng.random((pages, heads)) < 0.05, device=DEV)
    V[far] = 3e38
    say(f"  launch: decode_attention, some heads beyond fp32, beams {beams}")
    _check(randn(rng, (n, heads * d), BF16), K, V, tables, lens, beams=beams)


def test_the_small_end_of_bf16():
    """Values and keys down to the type's smallest numbers count for what they are."""
    rng = np.random.default_rng(5)
    lens, page, d = [40, 300], 16, 64
    tables, pages = paged(rng, lens, page)
    K = pool(rng, tables, lens, pages, 2, page, d, BF16)
    for std in (1e-35, 1e-37):
        V = pool(rng, tables, lens, pages, 2, page, d, BF16, std=std)
        _check(randn(rng, (2, 2 * d), BF16), K, V, tables, lens)


def _exactly(q, K, V, tables, lens, beams=1, **kw):
    """Heads that are all beyond fp32: computed in 64 bits, rounded to fp32 and to the output's type; what is no number
    is the definition's."""
    ro, rl = decode.attention(wide(q), wide(K), wide(V), tables, lens, float(np.float32(kw.get("scale", K.shape[3] ** -0.5))),
                              None if kw.get("slopes") is None else wide(kw["slopes"]))
    for t in (tables, _wider(tables, K.shape[2])):
        out, lse = i8.decode_attention(q, K, V, ints(t), ints(lens), beams=beams, **kw)
        torch.cuda.synchronize()
        o, s = wide(out), wide(lse)
        some = np.isfinite(ro)
        assert np.array_equal(o[~some], ro[~some], equal_nan=True)
        near(out[torch.as_tensor(some, device=DEV)], ro[some], 2.0 ** -23 * np.abs(ro[some]), "out")
        with np.errstate(over="ignore"):
            want = rl.astype(np.float32)
        some = np.isfinite(want)
        assert np.array_equal(s[~some], want[~some], equal_nan=True), (s[~some], want[~some])
        assert (np.abs(s[some] - rl[some]) <= 2.0 ** -23 * np.abs(rl[some])).all()
    return ro, rl


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_an_infinite_score(dtype):
    """One key's score is infinite: so is the logarithm of the sum, and the result is no number (nor are both beside a NaN)."""
    rng = np.random.default_rng(11)
    lens, page, d = [50, 300, 1, 700], 16, 64
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, 2, page, d, dtype) for _ in range(2))
    for i, n in enumerate(lens):
        K[int(tables[i, (n - 1) // page]), :, (n - 1) % page, 5] = float("inf")
    q = randn(rng, (4, 4 * d), dtype).abs()
    say(f"  launch: decode_attention, an infinite score, {dtype}")
    _, lse = _exactly(q, K, V, tables, lens)
    assert np.isposinf(lse).all()
    _exactly(q, K, V, tables, lens, beams=2)
    K[int(tables[1, 0]), 1, 3, 0] = float("nan")
    _, lse = _exactly(q, K, V, tables, lens)
    assert np.isnan(lse[1, 2:]).all() and np.isposinf(lse[1, :2]).all()


@pytest.mark.parametrize("beams", [1, 2])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scores_of_minus_infinity(dtype, beams):
    """A key of score -inf has no weight beside others; where all are, the log-sum is -inf and the result no number. A
    sequence without tokens still gives 0."""
    rng = np.random.default_rng(12)
    lens, page, d, heads = [1, 40, 300, 700, 0, 33], 16, 64, 2
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, heads, page, d, dtype) for _ in range(2))
    q = randn(rng, (6, 2 * heads * d), dtype).abs()
    for i in (0, 2):
        K[ints(tables[i][tables[i] >= 0]).long(), :, :, 7] = float("-inf")
    say(f"  launch: decode_attention, scores of -inf, {dtype}, beams {beams}")
    ro, rl = _exactly(q[[0, 2]], K, V, tables[[0, 2]], [1, 300], beams=beams)
    assert np.isneginf(rl).all() and np.isnan(ro).all()
    for i, n in ((1, 40), (3, 700)):                  # all tokens but two
        at = rng.choice(n, size=n - 2, replace=False)
        K[ints(tables[i, at // page]).long(), :, ints(at % page).long(), 7] = float("-inf")
    _exactly(q[[1, 3]], K, V, tables[[1, 3]], [40, 700], beams=beams)
    out, lse = i8.decode_attention(q, K, V, ints(tables), ints(lens), beams=beams)
    assert not out[4].any() and torch.isneginf(lse[4]).all() and torch.isfinite(out[5]).all()


@pytest.mark.parametrize("beams", [1, 2])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_finite_scores_that_fp32_has_no_room_for(sign, beams):
    """bf16's queries and keys are finite and their products are not in fp32, above and below; the largest score takes the
    weight, equal ones share it, and the log-sum is what fp32 makes of it."""
    rng = np.random.default_rng(13)
    lens, page, d, heads = [1, 40, 700, 5], 16, 64, 2
    tables, pages = paged(rng, lens, page)
    K, V = pool(rng, tables, lens, pages, heads, page, d, BF16, std=0.0), pool(rng, tables, lens, pages, heads, page, d, BF16)
    q = torch.full((4, 2 * heads * d), 1e20, dtype=BF16, device=DEV)
    say(f"  launch: decode_attention, scores beyond fp32, sign {sign}, beams {beams}")
    for i, n in enumerate(lens):                      # equal scores
        K[ints(tables[i][tables[i] >= 0]).long()] += sign * 1e20
    ro, rl = _exactly(q, K, V, tables, lens, beams=beams)
    assert np.isfinite(ro).all() and (np.abs(rl) > 1e39).all()
    # scores far apart: that of one key is the largest
    for i, n in enumerate(lens):
        for j in range(n):
            K[int(tables[i, j // page]), :, j % page] *= 1.0 + (j != n // 2) * (1 if sign < 0 else -1) * (0.25 + 0.5 * rng.random())
    ro, _ = _exactly(q, K, V, tables, lens, beams=beams)
    for i, n in enumerate(lens):
        v = wide(V[int(tables[i, n // 2 // page]), :, n // 2 % page]).reshape(-1)
        assert np.array_equal(ro[i].reshape(heads, 2, d)[:, 0].reshape(-1), v)


def test_sums_that_leave_fp32_on_the_way():
    """Products of +-2e38 whose sum is a number of fp32, in orders of which any partial sum may be beyond it."""
    page, d = 16, 16
    q = torch.ones((1, d), dtype=BF16, device=DEV)
    big = float(torch.tensor(2e38, dtype=BF16))
    say("  launch: decode_attention, partial sums beyond fp32")
    for order in range(6):
        rng = np.random.default_rng(order)
        K = torch.zeros((1, 1, page, d), dtype=BF16, device=DEV)
        V = randn(rng, (1, 1, page, d), BF16)
        # the sums: 3, -2e38 (which is the largest in the second call), 5
        for j, row in enumerate(([big, big, -big, -big, 3.0], [-big, -big, big], [big, -big, 5.0])):
            place = rng.permutation(d)[:len(row)]
            K[0, 0, j, torch.as_tensor(place, device=DEV)] = torch.tensor(row, dtype=BF16, device=DEV)
        out, lse = i8.decode_attention(q, K, V, ints([[0]]), ints([3]), scale=1.0)
        # A sum of terms of 2e38 is off by up to (d + 4) 2^-24 * 8e38 = 1e33 in fp32, and by 1e24 in 64 bits, so which of 3
        # and 5 is the larger is not determined, nor are the weights but for their being weights: the result lies between
        # the values (beside the roundings of weights and result), and the log-sum within 1e33 of the definition's
        v = wide(V)[0, 0, :3]
        slack = 2.0 ** -7 * np.abs(v).max(0)
        assert (wide(out)[0] >= v.min(0) - slack).all() and (wide(out)[0] <= v.max(0) + slack).all()
        assert abs(float(lse)) <= 1e33
        K[0, 0, 0] = -big                             # -3.2e39, -2e38
        out, lse = i8.decode_attention(q, K, V, ints([[0]]), ints([2]), scale=1.0)
        assert np.array_equal(wide(out)[0], wide(V)[0, 0, 1]) and abs(float(lse) + big) <= 2.0 ** -23 * big


def test_a_scale_or_bias_beyond_fp32():
    rng = np.random.default_rng(14)
    lens, page, d = [1, 3, 300], 16, 64
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, 2, page, d, F16) for _ in range(2))
    q = randn(rng, (3, 2 * d), F16, 30.0)
    say("  launch: decode_attention, scales and biases beyond fp32")
    for scale in (3e38, -3e38):
        _exactly(q, K, V, tables, lens, scale=scale)
    _exactly(q, K, V, tables, lens, slopes=torch.tensor([3e38, -3e38], device=DEV))


@pytest.mark.parametrize("beams", [1, 3])
def test_captured_and_replayed_beyond_fp32_and_back(beams):
    """One graph, replayed over values that leave fp32's range in some heads, in none, in scores, and on another stream:
    the eager call's result each time, and the same one twice."""
    rng = np.random.default_rng(15)
    lens, page, d, heads = [200, 7, 700, 33, 0, 128], 16, 64, 4
    tables, pages = paged(rng, lens, page)
    tables = _wider(tables, page)
    K, V = (torch.zeros((pages, 2, page, d), dtype=BF16, device=DEV) for _ in range(2))
    q, t, n = torch.zeros((6, heads * d), dtype=BF16, device=DEV), ints(tables), ints(lens)
    out, lse = torch.empty_like(q), torch.empty((6, heads), device=DEV)
    ws = torch.empty(i8.decode_attention_workspace(6, heads, 2, d), dtype=torch.uint8, device=DEV)
    say(f"  launch: decode_attention beyond fp32, captured, beams {beams}")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i8.decode_attention(q, K, V, t, n, out=out, lse=lse, beams=beams, workspace=ws)
    side = torch.cuda.Stream()
    for step in range(6):
        k, v = (pool(rng, tables, lens, pages, 2, page, d, BF16) for _ in range(2))
        if step % 3 == 0:
            v[::3, 1] = 3e38
        if step % 3 == 1:
            k[::2, 0] *= 1e30
        x = randn(rng, (6, heads * d), BF16, 1e12 if step == 4 else 1.0)
        for a, b in ((K, k), (V, v), (q, x)):
            a.copy_(b)
        ws.random_(0, 255)
        g.replay()
        eager = i8.decode_attention(q, K, V, t, n, beams=beams)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = i8.decode_attention(q, K, V, t, n, beams=beams)
        torch.cuda.synchronize()
        assert torch.isfinite(out).all()
        for a, b in (eager, other):
            assert torch.equal(out, a) and torch.equal(lse, b)
