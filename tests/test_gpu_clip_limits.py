"""Clipping at the ends: infinities and NaN beside every kind of limit, and
factors that fp32 does not hold. Bounds: as test_gpu_clip.py, with one rounding
more of the product (3 e relative beside the output's half ulp)."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import EPS32, near, randn, wide
from gpu_util import say
from oracle import adapt

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm", [INF, 0.0, 1.0])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_not_finite_gradients(bad, max_norm, in_place):
    """A NaN makes everything NaN. An infinity gives a factor of 0, or of 1 if
    nothing is to be clipped: then no gradient changes."""
    rng = np.random.default_rng(3)
    g = [randn(rng, 100, F32), randn(rng, (33, 21), BF16), randn(rng, 20000, F16)]
    g[1][7, 7] = bad
    before = [t.clone() for t in g]
    out = g if in_place else [torch.empty_like(t) for t in g]
    say(f"  launch: clip_grad_norm with {bad}, limit {max_norm}, in place {in_place}")
    total = float(i8.clip_grad_norm(g, max_norm, out=None if in_place else out))
    ref_total, ref = adapt.clip_grad_norm([wide(t) for t in before], max_norm)
    if np.isnan(bad):
        assert np.isnan(total) and np.isnan(ref_total) and all(torch.isnan(t).all() for t in out)
        assert all(np.isnan(r).all() for r in ref)
        return
    assert total == INF and ref_total == INF
    for t, r, b in zip(out, ref, before):
        assert np.array_equal(wide(t), r, equal_nan=True)
        if max_norm == INF:
            assert torch.equal(t, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size,max_norm", [(1e30, 1e-10), (1e36, 1e-10), (1e36, 1e-30), (1e30, 1e-38)])
def test_factors_beyond_fp32(size, max_norm, dtype):
    """max_norm / N below fp32's normal numbers, or below all of them: the
    products are numbers that fp32 holds."""
    rng = np.random.default_rng(4)
    g = [randn(rng, 70, dtype, size), randn(rng, (31, 33), dtype, size)]
    say(f"  launch: clip_grad_norm of values near {size} to {max_norm} {dtype}")
    out = [torch.empty_like(t) for t in g]
    i8.clip_grad_norm(g, max_norm, out=out)
    torch.cuda.synchronize()
    _, ref = adapt.clip_grad_norm([wide(t) for t in g], float(np.float32(max_norm)))
    for o, r in zip(out, ref):
        near(o, r, 3 * EPS32 * np.abs(r), "out")
