"""Layer norm of more rows than one launch takes: a dimension of a grid has
fewer than 2^32 threads, and a row takes 64 of them or more."""

import pytest
import torch

import int8_quantized_matmul_amd as i8
from gpu_util import DEV, say
from test_gpu_layer_norm import _check_backward, _check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_more_rows_than_a_launch_takes(in_place):
    s, h = 2 ** 26 + 77, 3
    say(f"  launch: layer_norm s={s} h={h}")
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn((s, h), generator=g, device=DEV, dtype=torch.float16)
    w, b = torch.tensor([1.0, 2.0, -1.0], device=DEV), torch.tensor([0.0, 0.5, 1.0], device=DEV)
    at = torch.cat([torch.arange(k, k + 50, device=DEV) for k in (0, 2 ** 25 - 25, 2 ** 26 - 25, s - 50)])
    rows = X[at]
    Z = X.clone() if in_place else X
    Y = Z if in_place else torch.full_like(X, float("nan"))
    mean, rstd = (torch.full((s,), float("nan"), device=DEV) for _ in range(2))
    i8.layer_norm(Z, w, b, 1e-3, Y=Y, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    _check_forward(rows, w, b, 1e-3, Y[at], mean[at], rstd[at])
    assert bool(torch.isfinite(mean).all()) and bool(torch.isfinite(rstd).all()) and bool(torch.isfinite(Y).all())
    if in_place:
        return
    dX = torch.full_like(X, float("nan"))
    i8.layer_norm_backward(Y, X, w, mean, rstd, dX=dX)
    torch.cuda.synchronize()
    _check_backward(Y[at], rows, w, mean[at], rstd[at], dX[at], None, None)
    assert bool(torch.isfinite(dX).all())
