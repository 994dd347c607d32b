"""Row quantisers, detection, the forward and the outlier product for more
rows than one launch takes: a dimension of a grid has fewer than 2^32 threads,
and a row takes a wavefront. Runs of rows at the beginning, around every
power of two that a launch may end at, and at the end are compared with calls
on those rows alone, bit for bit.
"""

import pytest
import torch

import int8_quantized_matmul_amd as i8
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

S, H = 2 ** 26 + 301, 64
PADDED = 32                                 # columns of X_O that one outlier column has written
RUNS = [slice(0, 300)] + [slice(2 ** k - 150, 2 ** k + 150) for k in (22, 23, 24, 25, 26)] + [slice(S - 300, S)]


@pytest.fixture(scope="module")
def rows():
    """X with one outlier column, found in the last row alone, and the largest
    value below the threshold beyond 2^26 rows."""
    g = torch.Generator(device=DEV).manual_seed(5)
    X = torch.randn((S, H), generator=g, device=DEV, dtype=torch.float16).clamp_(-4, 4)
    X[S - 1, 17] = 9.0
    X[2 ** 26 + 5, 40] = -5.5
    say(f"  launch: detect_outlier_cols s={S}")
    found = i8.detect_outlier_cols(X)
    torch.cuda.synchronize()
    assert int(found[2]) == 1 and int(found[1][0]) == 17
    yield X, found
    torch.cuda.empty_cache()


@pytest.mark.parametrize("scheme", ["rowwise", "rowwise_zeropoint"])
def test_row_quantisers(rows, scheme):
    X, found = rows
    call = getattr(i8, f"quantize_{scheme}")
    say(f"  launch: quantize_{scheme} s={S}")
    got = call(X, *found)
    for r in RUNS:
        some = call(X[r].contiguous(), *found)
        torch.cuda.synchronize()
        for a, b in zip(got[:-1], some[:-1]):
            assert torch.equal(a[r], b)
        assert torch.equal(got[-1][r, :PADDED], some[-1][:, :PADDED])


def test_tensorwise(rows):
    X, found = rows
    say(f"  launch: quantize_tensorwise s={S}")
    Xq, c_x, X_O = i8.quantize_tensorwise(X, *found)
    torch.cuda.synchronize()
    assert bool((c_x == torch.tensor(127.0, device=DEV) / 5.5).all())
    # the same constant comes out of any rows beside the one with the largest value
    last = X[2 ** 26 + 5:2 ** 26 + 6]
    for r in RUNS:
        some, _, out = i8.quantize_tensorwise(torch.cat([X[r], last]).contiguous(), *found)
        torch.cuda.synchronize()
        assert torch.equal(Xq[r], some[:-1]) and torch.equal(X_O[r, :PADDED], out[:-1, :PADDED])


def test_forward(rows):
    X, found = rows
    g = torch.Generator(device=DEV).manual_seed(6)
    W = (0.1 * torch.randn((H, 64), generator=g, device=DEV)).half()
    Wq, c_w = i8.quantize_colwise_weights(W)
    say(f"  launch: forward s={S}")
    C = i8.forward(X, Wq, c_w, W)
    torch.cuda.synchronize()
    last = X[S - 1:S]
    for r in RUNS:                          # the outlier's row, so that the same column is one
        some = i8.forward(torch.cat([X[r], last]).contiguous(), Wq, c_w, W)
        torch.cuda.synchronize()
        assert torch.equal(C[r], some[:-1])


def test_outlier_product():
    s, o = 2 ** 24 + 100, 1024              # a wavefront for each 16 x 16 outputs: more than 2^32 threads
    g = torch.Generator(device=DEV).manual_seed(7)
    W = (0.1 * torch.randn((H, o), generator=g, device=DEV)).half()
    X_O = torch.zeros((s, i8.x_o_stride(H)), dtype=torch.float16, device=DEV)
    X_O[:, :3] = torch.randn((s, 3), generator=g, device=DEV, dtype=torch.float16)
    idx = torch.zeros(H, dtype=torch.int32, device=DEV)
    idx[:3] = torch.tensor([3, 17, 60])
    n = torch.tensor([3], dtype=torch.int32, device=DEV)
    C = torch.full((s, o), float("nan"), device=DEV)
    say(f"  launch: outlier_matmul s={s} o={o}")
    i8.outlier_matmul(X_O, idx, n, W, C)
    torch.cuda.synchronize()
    for r in (slice(0, 300), slice(2 ** 23 - 150, 2 ** 23 + 150), slice(2 ** 24 - 150, 2 ** 24), slice(s - 300, s)):
        assert torch.equal(C[r], i8.outlier_matmul(X_O[r].contiguous(), idx, n, W))
    del C
    torch.cuda.empty_cache()
