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
