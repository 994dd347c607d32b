"""Beam search's selection against its definition in 64 bits.

Bounds: a row's sum of exponentials is a chain of at most vocab / 512 + 20
additions in fp32 of terms that are off by 2^-21 at most (the exponential's
argument x - m, at most 100 in size where the term matters, is rounded to 2^-24
of itself, twice; the exponential to 2^-23), so its logarithm is off by
(vocab / 512 + 20) 2^-24 + 2^-21 + 2^-17 in the worst case of all terms 100 below the
largest; the score itself is rounded to fp32. Two continuations whose scores
lie nearer than twice that may change places; all others may not."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import randn, strided, wide
from decode_util import ints
from gpu_util import DEV, say
from oracle import decode

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _check(logits, scores, k, history=None, **kw):
    got = i8.beam_select(logits, scores, k, history, **kw)
    torch.cuda.synchronize()
    n, beams = scores.shape
    x, V = wide(logits), logits.shape[1]
    rs, rp, rt, rh = decode.select(x, wide(scores), k, None if history is None else history.cpu().numpy())
    s, p, t = wide(got[0]), got[1].cpu().numpy(), got[2].cpu().numpy()
    off = (V / 512 + 20) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -17
    assert np.array_equal(np.isneginf(s), np.isneginf(rs))
    there = ~np.isneginf(rs)
    limit = off + 2.0 ** -23 * np.abs(np.where(there, rs, 0))
    assert (np.abs(s - rs)[there] <= limit[there]).all(), np.abs(s - rs)[there].max()
    differ = (p != rp) | (t != rt)
    if differ.any():                                  # only among continuations that lie within the bound
        x3 = x.reshape(n, beams, V)
        top = x3.max(2)
        lse = top + np.log(np.exp(x3 - top[:, :, None]).sum(2))
        for b, i in np.argwhere(differ):
            mine = float(scores[b, p[b, i] - b * beams]) + x[p[b, i], t[b, i]] - lse[b, p[b, i] - b * beams]
            assert abs(mine - rs[b, i]) <= 2 * limit[b, i], (b, i, mine, rs[b, i])
        assert all(len(set(zip(p[b], t[b]))) == k for b in range(n))
    if history is not None:
        want = np.concatenate([history.cpu().numpy()[p.reshape(-1)], t.reshape(-1, 1)], 1)
        assert np.array_equal(got[3].cpu().numpy(), want)
    else:
        assert got[3] is None
    return got, differ


CASES = [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 50257, 4), (3, 2, 511, 64), (2, 64, 513, 64), (5, 5, 2049, 10), (1, 1, 250000, 50),
         (7, 3, 1000, 6), (64, 4, 3001, 8), (1, 8, 129, 16), (300, 2, 70, 2), (2, 64, 1, 64), (1, 16, 30000, 33)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,beams,V,k", CASES)
def test_against_the_definition(n, beams, V, k, dtype):
    rng = np.random.default_rng(n + beams + V)
    logits = randn(rng, (n * beams, V), dtype, 3.0)
    scores = torch.from_numpy(rng.uniform(-9, 0, size=(n, beams)).astype(np.float32)).to(DEV)
    history = ints(rng.integers(0, V, size=(n * beams, k % 5 * 40)))
    say(f"  launch: beam_select {n} x {beams} x {V}, k {k}, {dtype}")
    _, differ = _check(logits, scores, k, history)
    assert not differ.any() or V > 20000 or n > 50
    _check(strided(logits, 3, 1), scores, k, strided(history.float(), 5).int() if history.shape[1] else None)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_ties_go_to_the_lowest(dtype):
    """Equal logits, within a row, over its parts and over beams with equal scores: beam after beam, token after token."""
    V, beams = 5000, 4
    logits = torch.zeros((2 * beams, V), dtype=dtype, device=DEV)
    scores = torch.zeros((2, beams), device=DEV)
    say(f"  launch: beam_select, ties, {dtype}")
    _, differ = _check(logits, scores, 64)
    assert not differ.any()
    logits[:, 17::613] = 2.0                          # in every beam the same nine, over many parts
    _, differ = _check(logits, scores, 30)
    assert not differ.any()
    logits[:, 4999], logits[:, 0] = 5.0, 5.0
    _, differ = _check(logits, scores, 9)
    assert not differ.any()
    x = torch.arange(V, device=DEV) % 7               # many ties at every level
    _, differ = _check(x.to(dtype).expand(2 * beams, V).contiguous(), scores, 64)
    assert not differ.any()


def test_ascending_and_descending_logits():
    V = 30011
    up = torch.linspace(-30, 5, V, device=DEV)
    logits = torch.stack([up, up.flip(0), up, up.flip(0)])
    say("  launch: beam_select, ascending and descending")
    for k in (1, 5, 64):
        _, differ = _check(logits, torch.tensor([[-1.0, -1.7], [0.0, -40.0]], device=DEV), k)
        assert not differ.any()


@pytest.mark.parametrize("k", [1, 31, 33, 64])
def test_best_in_one_place(k):
    """All that is chosen lies together, anywhere in rows of several steps, rising, falling or of few different values."""
    V, rows = 20011, 512                              # two parts a row
    rng = np.random.default_rng(k)
    x = rng.integers(-40, 0, size=(rows, V)).astype(np.float32) / 8
    for r in range(rows):
        at = [0, 500, 1000, 2490, 9980, 10010, V - 130, V - k][r % 8]
        size = min(V - at, 130) if r % 3 else min(V - at, k)
        x[r, at:at + size] = [np.arange(size) / 16, -np.arange(size) / 16 + 9, np.arange(size) // 40, np.zeros(size)][r // 8 % 4] + 1
    logits = torch.from_numpy(x).to(DEV)
    scores = torch.zeros(rows, 1, device=DEV)
    say(f"  launch: beam_select {rows} x 1 x {V}, k {k}")
    got = i8.beam_select(logits, scores, k)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    assert np.array_equal(got[2].cpu().numpy(), order)
    _check(logits[:24], scores[:24], k)


def test_what_leaves_nothing():
    """Masked tokens (-inf and the type's lowest value), beams that have ended (a score of -inf), rows without a token left,
    NaN and +inf logits, scores that are not finite."""
    rng = np.random.default_rng(2)
    V, inf, nan = 700, float("inf"), float("nan")
    logits = randn(rng, (6 * 3, V), F16, 2.0)
    logits[0, 5:] = -inf                              # five tokens left
    logits[1] = -inf
    logits[2, 100:] = -65504.0
    logits[3, 3], logits[4, 699] = nan, inf
    logits[6:9] = -inf
    logits[9, 1:], logits[10], logits[11] = -inf, nan, -inf
    logits[15, ::2] = -inf
    scores = torch.tensor([[0, -1, -2], [-1, -1, -1], [0, 0, 0], [-3, -3, -3], [0, -inf, -inf], [-1, nan, inf]], device=DEV)
    say("  launch: beam_select, masked")
    for k in (1, 3, 6, 64):
        _, differ = _check(logits, scores, k)
        assert not differ.any()
    s, p, t, _ = i8.beam_select(logits, scores, 3)
    assert p[2].tolist() == [6, 6, 6] and t[2].tolist() == [0, 1, 2] and torch.isneginf(s[2]).all()
    # the first step of a search: all beams alike, only the first counts
    s, p, t, _ = i8.beam_select(logits[12:15], torch.tensor([[0.0, -inf, -inf]], device=DEV), 3)
    assert p.tolist() == [[0, 0, 0]] and len(set(t[0].tolist())) == 3


def test_large_and_far_apart():
    rng = np.random.default_rng(3)
    logits = randn(rng, (4, 4000), F32, 1.0) * torch.tensor([[1e-6], [1e4], [1e30], [1.0]], device=DEV)
    logits[3] += 3e4
    say("  launch: beam_select, large logits")
    _check(logits, torch.tensor([[-1e3, 0.0, 5.0, -1e30]], device=DEV), 12)
    _check(logits[3:], torch.zeros((1, 1), device=DEV), 40)


def test_same_every_time_streams_and_outputs():
    rng = np.random.default_rng(4)
    logits, scores, h = randn(rng, (12, 9000), F16, 2.0), torch.zeros((3, 4), device=DEV), ints(rng.integers(0, 9, size=(12, 3)))
    say("  launch: beam_select, repeated")
    first = i8.beam_select(logits, scores, 8, h)
    outs = dict(scores_out=torch.empty((3, 8), device=DEV), parents=ints(np.zeros((3, 8))), tokens=ints(np.zeros((3, 8))),
                workspace=torch.empty(i8.beam_select_workspace(3, 4, 9000, 8), dtype=torch.uint8, device=DEV))
    store = ints(np.full((24, 9), -7))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        outs["workspace"].random_(0, 255)
        again = i8.beam_select(logits, scores, 8, h, history_out=store[:, 2:6], **outs)
        with torch.cuda.stream(side):
            other = i8.beam_select(logits, scores, 8, h)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, other))
        assert again[1].data_ptr() == outs["parents"].data_ptr() and (store[:, :2] == -7).all() and (store[:, 6:] == -7).all()


def test_captured_and_replayed():
    rng = np.random.default_rng(5)
    x, s, h = randn(rng, (6, 2000), BF16, 2.0), torch.zeros((2, 3), device=DEV), ints(rng.integers(0, 9, size=(6, 5)))
    say("  launch: beam_select, captured")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = i8.beam_select(x, s, 3, h)
    for _ in range(4):
        x.copy_(randn(rng, (6, 2000), BF16, 2.0))
        s.copy_(torch.rand((2, 3), device=DEV))
        g.replay()
        eager = i8.beam_select(x, s, 3, h)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_nothing_and_refusals():
    x, s = torch.zeros((6, 100), device=DEV), torch.zeros((2, 3), device=DEV)
    assert [v.shape[0] for v in i8.beam_select(x[:0], s[:0])[:3]] == [0, 0, 0]
    h = ints(np.zeros((6, 4)))
    for a in ((x[:5], s), (x.double(), s), (x.cpu(), s), (x, s.half()), (x, s, 3, h[:5]), (x, s, 3, h.long()), (x.t(), s)):
        with pytest.raises(ValueError):
            i8.beam_select(*a)
    for kw in (dict(k=0), dict(k=65), dict(k=301), dict(scores_out=s)):
        with pytest.raises(i8.I8MMError):
            i8.beam_select(x, s, **kw)
    with pytest.raises(i8.I8MMError):
        i8.beam_select(x[:, :2].contiguous()[:1], s[:1, :1].contiguous(), 3)
