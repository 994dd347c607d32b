"""Beam search's selection within the bound that its roundings give, and over more rows and requests than a launch has blocks.

A term exp(x - top) of a row's sum takes two exponentials (of x less the lane's maximum, of that less the row's), whose
arguments' sizes add up to top - x; an argument is rounded by the subtraction, by log2 e and by the product: 2.5 * 2^-24 of
itself. An exponential is off by 2^-23, a lane's maximum changes once a step at most and is joined twice (lanes, wavefronts).
Of additions, a lane has 16 a step, one and a product for each of its steps, then 6 over the lanes and 4 over the wavefronts
with a product each; the parts are joined in 64 bits. So with A the mean of top - x by weight the log-sum is off by
  2.5 * 2^-24 A + 2^-23 + (16 + 4 steps + 18) 2^-24,
and a score by half a step of fp32 more. Within a beam the order is that of the logits; continuations of two beams may
change places where they lie within the two log-sums' bounds."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import randn, wide
from decode_util import ints
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _steps(rows, V):
    parts = max(1, min(1024 // min(rows, 1024), -(-V // 2048)))
    return -(-V // (parts * 4 * 512)) + 1


def _check(logits, scores, k):
    s, p, t, _ = i8.beam_select(logits, scores, k)
    torch.cuda.synchronize()
    n, beams = scores.shape
    x, V = wide(logits), logits.shape[1]
    top = x.max(1, keepdims=True)
    w = np.exp(x - top)
    lse = top[:, 0] + np.log(w.sum(1))
    off = 2.5 * 2.0 ** -24 * (w * (top - x)).sum(1) / w.sum(1) + 2.0 ** -23 + (34 + 4 * _steps(n * beams, V)) * 2.0 ** -24
    total = (wide(scores).reshape(-1, 1) + (x - lse[:, None])).reshape(n, beams * V)
    best = np.argsort(-total, axis=1, kind="stable")[:, :k]
    rs = np.take_along_axis(total, best, 1)
    s, p, t = wide(s), p.cpu().numpy().astype(int), t.cpu().numpy().astype(int)
    mine = np.take_along_axis(total, (p - beams * np.arange(n)[:, None]) * V + t, 1)
    assert (np.abs(s - mine) <= off[p] + 2.0 ** -24 * np.abs(mine) + 2.0 ** -24 * off[p]).all(), np.abs(s - mine).max()
    theirs = best // V + beams * np.arange(n)[:, None]
    other = (theirs != p) | (best % V != t)
    assert (np.abs(mine - rs)[other] <= (off[p] + off[theirs])[other]).all()
    # within a beam: its best tokens in order
    for b in range(n):
        for i in np.unique(p[b]):
            got = t[b][p[b] == i]
            assert np.array_equal(got, np.argsort(-x[i], kind="stable")[:len(got)])
    return other


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,beams,V,k", [(1, 4, 50257, 4), (64, 8, 6000, 16), (4, 8, 50272, 32), (1, 1, 250000, 64), (2, 64, 3001, 64),
                                         (130, 8, 2049, 8)])
def test_scores_and_order_within_the_bound(n, beams, V, k, dtype):
    rng = np.random.default_rng(n + V)
    say(f"  launch: beam_select {n} x {beams} x {V}, k {k}, {dtype}")
    scores = torch.from_numpy(rng.uniform(-9, 0, size=(n, beams)).astype(np.float32)).to(DEV)
    _check(randn(rng, (n * beams, V), dtype, 3.0), scores, k)
    # a few likely tokens over a long tail, and all alike
    x = rng.normal(size=(n * beams, V)) * 2 - 6
    x[np.arange(n * beams)[:, None], rng.integers(0, V, size=(n * beams, 30))] += 12 * rng.random((n * beams, 30))
    _check(torch.from_numpy(x.astype(np.float32)).to(DEV).to(dtype), scores, k)
    _check(torch.full((n * beams, V), -3.0, dtype=dtype, device=DEV), scores, k)


@pytest.mark.parametrize("n,beams,V,k", [(70001, 1, 5, 3), (40000, 2, 17, 4), (66000, 3, 9, 27)])
def test_more_requests_than_blocks(n, beams, V, k):
    """Blocks that take several rows, and several requests, one after another. Values whose sums are exact in any order of
    additions: rows of 0 and of -inf, of which the log-sum is that of a count."""
    rng = np.random.default_rng(n)
    x = np.where(rng.random((n * beams, V)) < 0.6, 0.0, -np.inf).astype(np.float32)
    x[np.arange(n * beams), rng.integers(0, V, size=n * beams)] = 0.0
    scores = (-rng.integers(0, 40, size=(n, beams)) / 4).astype(np.float32)
    history = rng.integers(0, 99, size=(n * beams, 2))
    say(f"  launch: beam_select {n} x {beams} x {V}")
    s, p, t, h = i8.beam_select(torch.from_numpy(x).to(DEV), torch.from_numpy(scores).to(DEV), k, ints(history))
    torch.cuda.synchronize()
    total = (scores.reshape(-1, 1).astype(np.float64) + x - np.log((x == 0).sum(1, keepdims=True))).reshape(n, beams * V)
    best = np.argsort(-total, axis=1, kind="stable")[:, :k]
    rs = np.take_along_axis(total, best, 1)
    s, p, t = wide(s), p.cpu().numpy(), t.cpu().numpy()
    assert np.array_equal(np.isneginf(s), np.isneginf(rs))
    some = np.isfinite(rs)
    assert (np.abs(s[some] - rs[some]) <= 2.0 ** -23 * (1 + np.abs(rs[some]))).all()
    assert np.array_equal(p, best // V + beams * np.arange(n)[:, None]) and np.array_equal(t, best % V)
    assert np.array_equal(h.cpu().numpy(), np.concatenate([history[p.reshape(-1)], t.reshape(-1, 1)], 1))
