"""Layer norm and its gradients against their definitions in 64 bits.

Bounds (e = 2^-24; a sum of terms t_k whose longest chain of fp32 additions
has L links is off by at most L e sum|t_k|): a row's sums are taken by at
least 64 threads and a tree, L <= h / 64 + 16, so the mean is off by at most
L e mean|x|. The variance adds a relative L e + 4 e (the mean's own error
enters it squared), rstd half of that and 3 e for its operations. The
outputs follow by the product rule; each further operation adds e times its
value. Column sums over s rows have L <= s + 16.
"""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import EPS32, near, randn, strided, wide
from gpu_util import DEV, say
from oracle import adapt

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)]
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 63), (5, 64), (1, 12288), (17, 513), (4, 1000), (33, 768), (300, 129), (2, 4099),
          (9, 5120), (3, 16385), (2, 40001), (1, 70000), (600, 24)]


def _inputs(s, h, xt, wt, seed):
    rng = np.random.default_rng(seed)
    X = rng.normal(size=(s, h)) + 0.5 * rng.normal(size=(s, 1))
    X[:, rng.integers(0, h)] *= 15.0
    X = torch.from_numpy(X.astype(np.float32)).to(DEV).to(xt)
    return X, randn(rng, h, wt) + 1, randn(rng, h, wt), randn(rng, (s, h), xt, 0.01)


def _check_forward(X, w, b, eps, Y, mean, rstd):
    h = X.shape[1]
    x, ww = wide(X), wide(w)
    ref, m, r = adapt.layer_norm(x, ww, None if b is None else wide(b), eps)
    L = h / 64 + 16
    ax = np.abs(x).mean(axis=1)
    dm = L * EPS32 * ax
    dr = (L + 10) * EPS32 * r + 0.5 * r ** 3 * dm ** 2
    near(mean, m, dm, "mean")
    near(rstd, r, dr, "rstd")
    n = (x - m[:, None]) * r[:, None]
    dn = r[:, None] * (dm[:, None] + EPS32 * np.abs(x - m[:, None])) + np.abs(n) * (dr / r)[:, None] \
        + 2 * EPS32 * np.abs(n)
    bound = np.abs(ww) * dn + 3 * EPS32 * (np.abs(n * ww) + (0 if b is None else np.abs(wide(b))))
    near(Y, ref, bound, "Y")


def _check_backward(dY, X, w, mean, rstd, dX, dw, db):
    s, h = X.shape
    x, dy, ww, m, r = wide(X), wide(dY), wide(w), wide(mean)[:, None], wide(rstd)[:, None]
    rx, rw, rb = adapt.layer_norm_backward(dy, x, ww, m[:, 0], r[:, 0])
    L = h / 64 + 16
    g, n = dy * ww, (x - m) * r
    mean_g, mean_gn = np.abs(g).mean(axis=1, keepdims=True), np.abs(g * n).mean(axis=1, keepdims=True)
    # terms of size |g|, mean|g| and |n| mean|g n|, through at most 8 operations of their own
    bound = r * EPS32 * (8 * np.abs(g) + (L + 8) * mean_g + (L + 16) * np.abs(n) * mean_gn)
    near(dX, rx, bound, "dX")
    if dw is not None:
        near(dw, rw, (s + 20) * EPS32 * np.abs(dy * n).sum(axis=0), "d_weight")
        near(db, rb, (s + 16) * EPS32 * np.abs(dy).sum(axis=0), "d_bias")


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("s,h", SHAPES)
def test_forward_and_backward(s, h, xt, wt):
    say(f"  launch: layer_norm s={s} h={h} {xt} {wt}")
    X, w, b, dY = _inputs(s, h, xt, wt, 7 * s + h)
    Y, mean, rstd = i8.layer_norm(X, w, b, 1e-5)
    dX, dw, db = i8.layer_norm_backward(dY, X, w, mean, rstd)
    torch.cuda.synchronize()
    _check_forward(X, w, b, 1e-5, Y, mean, rstd)
    _check_backward(dY, X, w, mean, rstd, dX, dw, db)


@pytest.mark.parametrize("xt", [F16, BF16, F32])
@pytest.mark.parametrize("h,extra,offset", [(64, 8, 8), (64, 1, 0), (100, 3, 5), (4096, 8, 1), (5141, 11, 3)])
def test_strided_and_unaligned_rows(h, extra, offset, xt):
    """Rows of a wider buffer at any element offset; the rest of it holds NaN
    and is neither read nor written."""
    s = 19
    say(f"  launch: layer_norm strided h={h} extra={extra} offset={offset} {xt}")
    X, w, b, dY = _inputs(s, h, xt, xt, h + extra)
    Xs, dYs = strided(X, extra, offset), strided(dY, extra + 2, offset + 1)
    out = torch.full((s, h + extra), float("nan"), dtype=xt, device=DEV)
    Y, mean, rstd = i8.layer_norm(Xs, w, b, 1e-5, Y=out[:, extra:])
    dXo = torch.full((s, h + extra), float("nan"), dtype=xt, device=DEV)
    dX, dw, db = i8.layer_norm_backward(dYs, Xs, w, mean, rstd, dX=dXo[:, :h])
    torch.cuda.synchronize()
    assert torch.isnan(out[:, :extra]).all() and torch.isnan(dXo[:, h:]).all()
    _check_forward(X, w, b, 1e-5, Y, mean, rstd)
    _check_backward(dY, X, w, mean, rstd, dX, dw, db)


def test_optional_arguments_and_in_place():
    X, w, b, dY = _inputs(21, 1032, F16, F16, 5)
    say("  launch: layer_norm without bias, in place, frozen")
    Y, mean, rstd = i8.layer_norm(X, w, None, 1e-3)
    _check_forward(X, w, None, 1e-3, Y, mean, rstd)
    dX, dw, db = i8.layer_norm_backward(dY, X, w, mean, rstd, param_grads=False)
    assert dw is None and db is None
    _check_backward(dY, X, w, mean, rstd, dX, None, None)
    Z = X.clone()
    i8.layer_norm(Z, w, None, 1e-3, Y=Z)
    assert torch.equal(Z, Y)


@pytest.mark.parametrize("xt", [F16, BF16, F32])
def test_no_rows(xt):
    X, w = torch.empty((0, 96), dtype=xt, device=DEV), torch.ones(96, dtype=xt, device=DEV)
    say("  launch: layer_norm with no rows")
    Y, mean, rstd = i8.layer_norm(X, w, w)
    assert Y.shape == (0, 96) and mean.shape == (0,)
    dX, dw, db = i8.layer_norm_backward(X, X, w, mean, rstd)
    torch.cuda.synchronize()
    assert dX.shape == (0, 96) and not dw.any() and not db.any()


@pytest.mark.parametrize("xt", [F16, BF16, F32])
def test_constant_rows_and_large_offsets(xt):
    """A constant row has variance 0: Y is the bias. A mean far above the
    spread of the values: the variance is taken about the mean, so it keeps
    its digits."""
    h = 2000
    w, b = torch.ones(h, dtype=xt, device=DEV), torch.full((h,), 0.25, dtype=xt, device=DEV)
    X = torch.full((4, h), 3.0, dtype=xt, device=DEV)
    X[1] = 0
    X[2] = 512 + torch.arange(h, device=DEV).remainder(3).to(xt) * 4
    X[3] = X[2]
    say("  launch: layer_norm of constant rows")
    Y, mean, rstd = i8.layer_norm(X, w, b, 1e-5)
    assert bool((Y[:2] == 0.25).all()) and torch.equal(Y[2], Y[3])
    _check_forward(X, w, b, 1e-5, Y, mean, rstd)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nan_and_infinity_stay_in_their_row(bad):
    X, w, b, dY = _inputs(9, 777, BF16, F32, 3)
    Y0, mean0, rstd0 = i8.layer_norm(X, w, b)
    dX0, _, db0 = i8.layer_norm_backward(dY, X, w, mean0, rstd0)
    X[4, 100] = bad
    say("  launch: layer_norm with a bad row")
    Y, mean, rstd = i8.layer_norm(X, w, b)
    dX, dw, db = i8.layer_norm_backward(dY, X, w, mean, rstd)
    torch.cuda.synchronize()
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(Y[keep], Y0[keep]) and torch.equal(dX[keep], dX0[keep]) and torch.equal(db, db0)
    assert torch.isnan(Y[4]).all() and torch.isnan(dX[4]).all() and torch.isnan(dw).all()


def test_same_bits_on_every_call_and_on_other_streams():
    X, w, b, dY = _inputs(513, 4100, F16, F16, 11)
    Y0, mean, rstd = i8.layer_norm(X, w, b)
    ref = i8.layer_norm_backward(dY, X, w, mean, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("  launch: layer_norm on two streams")
    with torch.cuda.stream(side):
        got = i8.layer_norm_backward(dY, X, w, mean, rstd)
        Y1 = i8.layer_norm(X, w, b)[0]
    again = i8.layer_norm_backward(dY, X, w, mean, rstd)
    torch.cuda.synchronize()
    for a, c, d in zip(ref, got, again):
        assert torch.equal(a, c) and torch.equal(a, d)
    assert torch.equal(Y0, Y1)


def test_gradients_against_differences():
    """The slope of <dY, layer_norm(X)> along a direction, by central
    differences of the definition in 64 bits (step 1e-5: off by about 1e-10
    relative), against the kernel's gradients: fp32 in and out, so each is off
    by a few e of its terms; 1e-5 of the norms holds that for h = 513."""
    rng = np.random.default_rng(2)
    X, w, b, dY = _inputs(6, 513, F32, F32, 8)
    _, mean, rstd = i8.layer_norm(X, w, b, 1e-2)
    grads = i8.layer_norm_backward(dY, X, w, mean, rstd)
    at = [wide(X), wide(w), wide(b)]
    for k in range(3):
        v = rng.normal(size=at[k].shape)
        f = [np.sum(wide(dY) * adapt.layer_norm(*[a + t * v if j == k else a for j, a in enumerate(at)], 1e-2)[0])
             for t in (1e-5, -1e-5)]
        g = wide(grads[k])
        assert abs((f[0] - f[1]) / 2e-5 - np.sum(g * v)) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(v)


def test_many_rows_beyond_32_bit_offsets():
    """s h above 2^31 elements: the last rows are the ones that a 32-bit
    offset would lose."""
    s, h = 2 ** 19 + 5, 4104
    say(f"  launch: layer_norm s={s} h={h}")
    X = torch.zeros((s, h), dtype=F16, device=DEV)
    rng = np.random.default_rng(4)
    tail, w = randn(rng, (7, h), F16), randn(rng, h, F16)
    X[-7:] = tail
    Y, mean, rstd = i8.layer_norm(X, w, w)
    _check_forward(tail, w, w, 1e-5, Y[-7:], mean[-7:], rstd[-7:])
    dX, dw, db = i8.layer_norm_backward(Y, X, w, mean, rstd, dX=torch.empty_like(X))
    dt, _, _ = adapt.layer_norm_backward(wide(Y[-7:]), wide(tail), wide(w), wide(mean[-7:]), wide(rstd[-7:]))
    near(dX[-7:], dt, 1e-4 * np.abs(dt).max() * np.ones_like(dt), "dX of the last rows")


def test_refusals():
    X, w = torch.zeros((4, 64), dtype=F16, device=DEV), torch.ones(64, dtype=F16, device=DEV)
    st = torch.zeros(4, device=DEV)
    for call in (lambda: i8.layer_norm(X.cpu(), w), lambda: i8.layer_norm(X[0], w),
                 lambda: i8.layer_norm(X.double(), w), lambda: i8.layer_norm(X, w.to(BF16)),
                 lambda: i8.layer_norm(X, w[:32]), lambda: i8.layer_norm(X.t(), w[:4]),
                 lambda: i8.layer_norm(X, w, w.float()), lambda: i8.layer_norm(X, w, mean=st[:3]),
                 lambda: i8.layer_norm(X, w, Y=torch.zeros((4, 64), dtype=F32, device=DEV)),
                 lambda: i8.layer_norm(X[:1].expand(4, 64), w),
                 lambda: i8.layer_norm_backward(X[:3], X, w, st, st),
                 lambda: i8.layer_norm_backward(X, X, w, st.half(), st),
                 lambda: i8.layer_norm_backward(X.clone(), X, w, st, st,
                                                workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        i8.layer_norm([1.0], w)
    for call in (lambda: i8.layer_norm(X, w, eps=-1.0), lambda: i8.layer_norm(X, w, eps=float("nan")),
                 lambda: i8.layer_norm_backward(X.clone(), X, w, st, st, dX=X)):
        with pytest.raises(i8.I8MMError, match="status -1"):
            call()
