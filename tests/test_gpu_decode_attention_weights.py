"""Attention's weights keep more digits than the cache's type: where large values cancel, the result is as exact as fp32
sums make it.

Bound: decode_util.attention_bounds with fp32's half step for a weight's rounding instead of the type's, and the two parts
that a weight is multiplied in: what the first, rounded to the type (off by u of itself), leaves is rounded to the type
again, so u^2 of the weight is lost (2^-16 in bf16, 2^-22 in fp16)."""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import HALF_ULP, near, randn, wide
from decode_util import attention_bounds, ints, paged, pool
from gpu_util import say
from oracle import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,d,page", [(1, 1, 16, 16), (8, 2, 64, 16), (4, 4, 128, 32), (2, 1, 256, 16)])
def test_large_values_that_cancel(heads, kv, d, page, dtype):
    rng = np.random.default_rng(heads)
    lens = [2, 3, 5, 17, 300, 2, 4]
    tables, pages = paged(rng, lens, page)
    K, V = (pool(rng, tables, lens, pages, kv, page, d, dtype) for _ in range(2))
    for i, n in enumerate(lens):                      # + and - 1000 in turn
        for t in range(n):
            V[int(tables[i, t // page]), :, t % page] = 1000.0 if t % 2 else -1000.0
    q = randn(rng, (len(lens), heads * d), dtype, 0.02)
    scale = d ** -0.5
    ro, rl = decode.attention(wide(q), wide(K), wide(V), tables, lens, scale)
    bo, bl = attention_bounds(q, K, V, tables, lens, scale, None, torch.float32)
    bo = bo + HALF_ULP[dtype] ** 2 * 1000.0
    say(f"  launch: decode_attention, values that cancel, {heads} heads on {kv}, {d}, {dtype}")
    for width in (tables.shape[1], -(-1040 // page)):
        table = np.full((len(lens), width), -1, np.int32)
        table[:, :tables.shape[1]] = tables
        out, lse = i8.decode_attention(q, K, V, ints(table), ints(lens))
        torch.cuda.synchronize()
        near(out, ro, bo, "out")
        assert (np.abs(wide(lse) - rl) <= bl).all()
        one, _ = i8.decode_attention(q, K, V, ints(table), ints([1] * len(lens)))
        assert (wide(one) == -1000).all()
    assert bo.max() < 0.25                            # of values of 1000
