"""The adapters beside infinities: where the definition gives an infinity, so
do the kernels, of the same sign; NaN where it gives NaN; and what it gives as
finite is within 2^-8 of the largest finite value (test_gpu_lora.py has the
tight bounds). The definition is taken in 64 bits from the kernels' own T, so
that each product is compared by itself.
"""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, wide
from gpu_util import DEV, say
from oracle import adapt
from test_gpu_lora import BF16, F16, _case

pytestmark = pytest.mark.gpu

INF = float("inf")
# s, h, o, r, G, ids: few tokens; many, with the operands in registers, in LDS and read again for each tile
CASES = [(3, 128, 192, 1, 2, "mixed"), (40, 128, 192, 20, 2, "runs"), (300, 256, 320, 8, 2, "mixed"),
         (300, 256, 320, 1, 3, "runs"), (520, 320, 256, 40, 1, "one"), (600, 192, 128, 100, 2, "runs"),
         (270, 128, 576, 32, 3, "mixed"), (330, 576, 128, 64, 2, "runs"), (256, 128, 192, 70, 2, "mixed")]


def _same(got, ref, what):
    g = wide(got)
    for name, f in (("NaN", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        assert np.array_equal(f(g), f(ref)), f"{what}: {name} at {f(g).sum()} places instead of {f(ref).sum()}"
    ok = np.isfinite(ref)
    size = np.abs(ref[ok]).max() if ok.any() else 0.0
    bound = np.where(ok, 2.0 ** -8 * size, 0.0)
    near(torch.where(torch.from_numpy(ok).to(DEV), got, 0.0), np.where(ok, ref, 0.0), bound, what)


def _check(c, say_):
    say(say_)
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])
    torch.cuda.synchronize()
    ids, f = c["ids"].cpu().numpy(), wide(c["scale"])
    x, dy, A, B, base, gbase = (wide(c[k]) for k in ("X", "dY", "A", "B", "base", "gbase"))
    with np.errstate(all="ignore"):
        _same(T, adapt.lora_forward(x, A, B, ids, f, base)[1], "T")
        t = wide(T)
        y = base.copy()
        for g in range(len(A)):
            i = np.nonzero(ids == g)[0]
            y[i] += f[g] * (t[i] @ B[g])
        rx, ra, rb, _ = adapt.lora_backward(dy, x, t, A, B, ids, f, gbase)
    for got, ref, what in ((Y, y, "Y"), (dX, rx, "dX"), (dA, ra, "dA"), (dB, rb, "dB")):
        _same(got, ref, what)
    return Y, dX, dA, dB


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", CASES)
def test_infinite_weights(s, h, o, r, G, kind, dtype):
    """Some elements of A and B: the columns of Y and dX that they reach are
    infinite in every token of their adapter."""
    c = _case(s, h, o, r, G, kind, dtype, seed=7)
    c["A"][0, 0, 5], c["A"][0, r - 1, 70] = INF, -INF
    c["B"][0, 0, 3], c["B"][0, r - 1, 100], c["B"][G - 1, r // 2, o - 1] = -INF, INF, INF
    c["ids"][0] = 0
    Y, dX, _, _ = _check(c, f"  launch: lora with infinite weights s={s} r={r} {kind} {dtype}")
    assert torch.isinf(Y).any() or r > 1


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", CASES)
def test_infinite_inputs(s, h, o, r, G, kind, dtype):
    """Elements of B and dY and, apart from them, of X: dB and dA of their
    columns are infinite, the other columns finite."""
    c = _case(s, h, o, r, G, kind, dtype, seed=8)
    c["ids"][0] = 0
    d = dict(c, dY=c["dY"].clone())
    d["dY"][0, 9], d["dY"][s // 2, 40] = INF, -INF
    _, _, _, dB = _check(d, f"  launch: lora with infinite output gradients s={s} r={r} {kind} {dtype}")
    assert torch.isinf(dB[0, :, 9]).all()
    d = dict(c, X=c["X"].clone())
    d["X"][0, 9], d["X"][s - 1, 33] = -INF, INF
    _check(d, f"  launch: lora with infinite inputs s={s} r={r} {kind} {dtype}")
    d = dict(c, B=c["B"].clone())
    d["B"][0, :, 11] = INF
    Y, _, _, _ = _check(d, f"  launch: lora with an infinite column s={s} r={r} {kind} {dtype}")
    assert not torch.isfinite(Y[0, 11])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_an_infinity_times_a_factor_that_is_small_beside_others(dtype):
    """T far below the other tokens' of its rank, and below the other ranks' of
    its token, is still not 0 beside an infinity."""
    c = _case(40, 128, 192, 4, 1, "one", dtype, seed=9)
    T = torch.ones((40, 4), device=DEV)
    T[5] = -2.0 ** -60
    c["dY"][5, 17] = INF
    say(f"  launch: lora with a small factor beside an infinity {dtype}")
    _, _, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"])
    assert bool((dB[0, :, 17] == -INF).all()) and bool(torch.isfinite(dB[0, :, :17]).all())
