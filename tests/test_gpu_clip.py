"""Global gradient norm and clipping against the definition in 64 bits.

Bounds: the squares are summed in fp64, so the norm is off by fp32's last
rounding alone (2^-24, and 2^-40 for the sums). The factor is rounded to
fp32, the product to fp32 and then to the output's type: 2 e relative beside
the output's half ulp.
"""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import EPS32, near, randn, wide
from gpu_util import DEV, say
from oracle import adapt

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _check(grads, max_norm, total, outs):
    n, ref = adapt.clip_grad_norm([wide(g) for g in grads], max_norm)
    assert total.shape == (1,) and total.dtype == F32
    assert abs(float(total) - n) <= (2.0 ** -24 + 2.0 ** -40) * n
    for k, (o, r) in enumerate(zip(outs, ref)):
        near(o, r, 2 * EPS32 * np.abs(r), f"out[{k}]")


def _grads(sizes, types, seed, std=1e-2):
    rng = np.random.default_rng(seed)
    return [randn(rng, n, types[k % len(types)], std) for k, n in enumerate(sizes)]


CASES = [([1], [F32]), ([7], [F16]), ([(3, 5)], [BF16]), ([1, 0, 2, (0, 4), 33], [F16, F32]),
         ([(64, 129), 4099, 16384, 16385, 100000], [F32, F16, BF16]), ([300000], [F16]), ([(1000, 1003)], [F32]),
         ([17 + k for k in range(250)], [F32, BF16]), ([5] * 97, [F16]), ([2 ** 20 + 3, 1, 2 ** 20], [BF16, F32])]


@pytest.mark.parametrize("ratio", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("sizes,types", CASES, ids=[str(k) for k in range(len(CASES))])
def test_norm_and_clip(sizes, types, ratio):
    grads = _grads(sizes, types, len(sizes))
    n, _ = adapt.clip_grad_norm([wide(g) for g in grads], 1.0)
    max_norm = n / ratio
    say(f"  launch: clip_grad_norm of {len(grads)} tensors, ratio {ratio}")
    outs = [torch.full_like(g, float("nan")) for g in grads]
    before = [g.clone() for g in grads]
    total = i8.clip_grad_norm(grads, max_norm, out=outs)
    torch.cuda.synchronize()
    _check(grads, max_norm, total, outs)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    again = i8.clip_grad_norm(grads, max_norm)             # in place
    torch.cuda.synchronize()
    assert torch.equal(again, total) and all(torch.equal(a, b) for a, b in zip(grads, outs))
    if ratio == 0.5:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 0), (0, 1), (3, 5), (1, 1)])
def test_unaligned_views(a, b, dtype):
    """Gradients and outputs anywhere in flat buffers; their neighbours stay."""
    n = 70001
    rng = np.random.default_rng(1)
    flat, out = randn(rng, n + 16, dtype), torch.full((n + 16,), float("nan"), dtype=dtype, device=DEV)
    say(f"  launch: clip_grad_norm of a view at {a} into {b} {dtype}")
    total = i8.clip_grad_norm([flat[a:a + n]], 3.0, out=[out[b:b + n]])
    torch.cuda.synchronize()
    _check([flat[a:a + n]], 3.0, total, [out[b:b + n]])
    assert torch.isnan(out[:b]).all() and torch.isnan(out[b + n:]).all()


def test_empty_lists_zeros_and_limits():
    say("  launch: clip_grad_norm of nothing")
    assert float(i8.clip_grad_norm([], 1.0)) == 0.0
    assert float(i8.clip_grad_norm([torch.empty(0, device=DEV)], 1.0)) == 0.0
    z = torch.zeros(1000, device=DEV)
    assert float(i8.clip_grad_norm([z], 1.0)) == 0.0 and not z.any()
    g = _grads([5000], [F32], 3)
    keep = g[0].clone()
    total = i8.clip_grad_norm(g, float("inf"))
    _check([keep], float("inf"), total, g)
    assert torch.equal(g[0], keep)
    i8.clip_grad_norm(g, 0.0)
    assert not g[0].any()


def test_squares_beyond_fp32():
    """Values whose squares leave fp32's range at either end."""
    for v in (1e25, 1e-30):
        g = torch.full((3000,), v, device=DEV)
        out = [torch.empty_like(g)]
        say(f"  launch: clip_grad_norm of values {v}")
        total = i8.clip_grad_norm([g], 1e-9 * v, out=out)
        n = float(np.float32(v)) * 3000 ** 0.5
        assert abs(float(total) - n) <= 2e-7 * n
        _check([g], 1e-9 * v, total, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity(bad):
    g = _grads([100, 20000], [F32, F16], 5)
    g[1][777] = bad
    say(f"  launch: clip_grad_norm with {bad}")
    out = [torch.empty_like(t) for t in g]
    total = float(i8.clip_grad_norm(g, 1.0, out=out))
    if np.isnan(bad):
        assert np.isnan(total) and all(torch.isnan(t).all() for t in out)
    else:
        assert total == np.inf and torch.isnan(out[1][777])
        out[1][777] = 0
        assert not any(t.any() for t in out)


def test_same_bits_on_other_streams_and_in_replays():
    g = _grads([(300, 301), 5, 70000], [F32, F16, BF16], 6)
    ref = [torch.empty_like(t) for t in g]
    total = i8.clip_grad_norm(g, 0.5, out=ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in g]
    say("  launch: clip_grad_norm on a second stream")
    with torch.cuda.stream(side):
        t2 = i8.clip_grad_norm(g, 0.5, out=out)
    torch.cuda.synchronize()
    assert torch.equal(total, t2) and all(torch.equal(a, b) for a, b in zip(ref, out))
    graph = torch.cuda.CUDAGraph()
    say("  capture: clip_grad_norm")
    with torch.cuda.graph(graph):
        t3 = i8.clip_grad_norm(g, 0.5, out=out)
    for k in range(3):
        for t in [*out, t3]:
            t.fill_(float("nan"))
        i8.clip_grad_norm([ref[0].clone()], 1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(total, t3) and all(torch.equal(a, b) for a, b in zip(ref, out))


def test_beyond_32_bit_offsets():
    n = 2 ** 31 + 70001
    say(f"  launch: clip_grad_norm of {n} values")
    g = torch.zeros(n, dtype=F16, device=DEV)
    g[-3:] = 2.0
    g[5] = 2.0
    total = i8.clip_grad_norm([g], 2.0)
    torch.cuda.synchronize()
    assert float(total) == 4.0
    assert bool((g[-3:] == 1.0).all()) and float(g[5]) == 1.0 and float(g[-4]) == 0.0


def test_refusals():
    g = torch.zeros(8, device=DEV)
    for call in (lambda: i8.clip_grad_norm([g.cpu()], 1.0), lambda: i8.clip_grad_norm([g.double()], 1.0),
                 lambda: i8.clip_grad_norm([g[::2]], 1.0), lambda: i8.clip_grad_norm([g], 1.0, out=[]),
                 lambda: i8.clip_grad_norm([g], 1.0, out=[g.half()]),
                 lambda: i8.clip_grad_norm([g], 1.0, out=[torch.zeros(7, device=DEV)]),
                 lambda: i8.clip_grad_norm([g], 1.0, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        i8.clip_grad_norm([1.0], 1.0)
    for m in (-1.0, float("nan")):
        with pytest.raises(i8.I8MMError, match="status -1"):
            i8.clip_grad_norm([g], m)
