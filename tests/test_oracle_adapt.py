"""The 64-bit definitions of layer norm's and the adapters' gradients against
differences of their forward passes (CPU). Central differences with step t of
a function with third derivatives of size about 1 are off by t^2, and by
2^-53 / t from rounding: with t = 1e-5 both are near 1e-10 of values near 1
to 100, so 1e-7 of the gradient's norm is asked for.
"""

import numpy as np
import pytest

from oracle import adapt

STEP, TOL = 1e-5, 1e-7


def _slope(f, x, v):
    return (f(x + STEP * v) - f(x - STEP * v)) / (2 * STEP)


def _agrees(slope, grad, v):
    assert abs(slope - np.sum(grad * v)) <= TOL * np.linalg.norm(grad) * np.linalg.norm(v)


@pytest.mark.parametrize("s,h", [(1, 2), (3, 5), (7, 64), (2, 301)])
def test_layer_norm_gradients_against_differences(s, h):
    rng = np.random.default_rng(10 * s + h)
    X, dY = rng.normal(size=(s, h)) + 0.3, rng.normal(size=(s, h))
    w, b = rng.normal(size=h) + 1, rng.normal(size=h)
    eps = 1e-2
    _, mean, rstd = adapt.layer_norm(X, w, b, eps)
    dX, dw, db = adapt.layer_norm_backward(dY, X, w, mean, rstd)
    loss = lambda x, ww, bb: np.sum(dY * adapt.layer_norm(x, ww, bb, eps)[0])   # noqa: E731
    for _ in range(3):
        v, u = rng.normal(size=(s, h)), rng.normal(size=h)
        _agrees(_slope(lambda x: loss(x, w, b), X, v), dX, v)
        _agrees(_slope(lambda x: loss(X, x, b), w, u), dw, u)
        _agrees(_slope(lambda x: loss(X, w, x), b, u), db, u)


@pytest.mark.parametrize("s,h,o,r,G", [(1, 4, 3, 1, 1), (9, 16, 24, 3, 4), (20, 33, 17, 8, 2)])
def test_adapter_gradients_against_differences(s, h, o, r, G):
    rng = np.random.default_rng(s + h + o)
    X, dY, base = rng.normal(size=(s, h)), rng.normal(size=(s, o)), rng.normal(size=(s, o))
    A, B = rng.normal(size=(G, r, h)), rng.normal(size=(G, r, o))
    ids, scale = rng.integers(-1, G + 1, size=s), rng.uniform(0.5, 2, size=G)
    _, T = adapt.lora_forward(X, A, B, ids, scale, base)
    dX, dA, dB, _ = adapt.lora_backward(dY, X, T, A, B, ids, scale, None)
    loss = lambda x, a, b: np.sum(dY * adapt.lora_forward(x, a, b, ids, scale, base)[0])   # noqa: E731
    for _ in range(3):
        v = rng.normal(size=X.shape)
        _agrees(_slope(lambda x: loss(x, A, B), X, v), dX, v)
        v = rng.normal(size=A.shape)
        _agrees(_slope(lambda x: loss(X, x, B), A, v), dA, v)
        v = rng.normal(size=B.shape)
        _agrees(_slope(lambda x: loss(X, A, x), B, v), dB, v)


def test_rows_without_an_adapter_keep_their_base():
    X, base = np.ones((3, 4)), np.arange(15.0).reshape(3, 5)
    A, B = np.ones((2, 2, 4)), np.ones((2, 2, 5))
    Y, T = adapt.lora_forward(X, A, B, np.array([-1, 1, 2]), np.array([1.0, 0.5]), base)
    assert np.array_equal(Y[[0, 2]], base[[0, 2]]) and not T[[0, 2]].any()
    assert np.array_equal(T[1], [4, 4]) and np.array_equal(Y[1], base[1] + 4)


def test_clip_grad_norm_worked_example():
    total, out = adapt.clip_grad_norm([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert total == 5.0 and abs(out[0][0] - 0.6) < 1e-6 and abs(out[1][0, 0] - 0.8) < 1e-6
    total, out = adapt.clip_grad_norm([np.array([3.0, 4.0])], 5.1)
    assert np.array_equal(out[0], [3.0, 4.0])
