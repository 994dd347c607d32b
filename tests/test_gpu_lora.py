"""Low-rank adapters and their gradients against their definitions in 64 bits.

Bounds (e = 2^-24): a product's sum over len terms is taken in steps of at
most 32 products and joined over at most 64 pieces, so its longest chain of
fp32 additions has at most len / 32 + 96 links, each off by e of the terms'
absolute sum (T, dT and the gradients of A and B). Where an fp32 factor (T,
dT) enters a product with 16-bit values it may be carried as a sum of 16-bit
parts: 2^-20 of the largest factor it is grouped with for fp16 (two parts),
2^-15 for bf16 in Y and dX (two parts, results of 8 bits), 2^-20 in the fp32
gradients (three parts). Y and dX are then rounded once.
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


def _ids(rng, s, G, kind):
    if kind == "one":
        ids = np.full(s, G - 1)
    elif kind == "none":
        ids = np.full(s, -1)
    elif kind == "runs":
        ids = np.sort(rng.integers(-1, G, size=s))[::-1].copy()
    elif kind == "mixed":
        ids = rng.integers(-1, G, size=s)
    else:                                # ids that name no adapter, of every sort
        ids = rng.choice(np.array([-2 ** 31, -5, -1, 0, G - 1, G, G + 3, 2 ** 31 - 1]), size=s)
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def _case(s, h, o, r, G, kind, dtype, seed=0):
    rng = np.random.default_rng([s, h, o, r, G, seed])
    c = dict(X=randn(rng, (s, h), dtype), A=randn(rng, (G, r, h), dtype, h ** -0.5), B=randn(rng, (G, r, o), dtype, 0.1),
             ids=_ids(rng, s, G, kind), base=randn(rng, (s, o), dtype), dY=randn(rng, (s, o), dtype, 1e-3),
             gbase=randn(rng, (s, h), dtype, 1e-3))
    c["scale"] = torch.from_numpy(rng.uniform(0.25, 4, size=G).astype(np.float32)).to(DEV)
    return c


def _per_row(c, P):
    """[s, len] rows of P [G, ...] by id, 0 where there is none."""
    ids = c["ids"].cpu().numpy()
    ok = (ids >= 0) & (ids < P.shape[0])
    out = np.zeros((len(ids),) + P.shape[1:])
    out[ok] = P[ids[ok]]
    return out


def _links(n):
    return (n / 32 + 96) * EPS32


def _dots(z, M, ids, G):
    """Absolute sums: sum_j |z_ij M_g[k, j]| for each row's adapter."""
    out = np.zeros((z.shape[0], M.shape[1]))
    for g in range(G):
        i = np.nonzero(ids == g)[0]
        out[i] = np.abs(z[i]) @ np.abs(M[g]).T
    return out


def _add_bound(P, dP, M, ids, factor, parts):
    """Bound of factor_i P_i M_g where P_i is off by dP_i."""
    out = np.zeros((P.shape[0], M.shape[2]))
    top = np.abs(P).max(axis=1, keepdims=True) if P.shape[1] else 0
    off = dP + parts * top + _links(P.shape[1]) * np.abs(P)
    for g in range(M.shape[0]):
        i = np.nonzero(ids == g)[0]
        out[i] = np.abs(factor[i, None]) * (off[i] @ np.abs(M[g]))
    return out


def _check_forward(c, Y, T, base):
    ids, G = c["ids"].cpu().numpy(), c["A"].shape[0]
    x, A, B, f = wide(c["X"]), wide(c["A"]), wide(c["B"]), wide(c["scale"])
    ry, rt = adapt.lora_forward(x, A, B, ids, f, None if base is None else wide(base))
    dt = _links(x.shape[1]) * _dots(x, A, ids, G)
    if T is not None:
        near(T, rt, dt, "T")
    parts = 2.0 ** -20 if Y.dtype == F16 else 2.0 ** -15
    bound = _add_bound(rt, dt, B, ids, _per_row(c, f), parts) + 2 * EPS32 * np.abs(ry)
    near(Y, ry, bound, "Y")
    if base is not None:
        none = (ids < 0) | (ids >= G)
        assert torch.equal(Y[torch.from_numpy(none)], base[torch.from_numpy(none)])


def _check_backward(c, T, dX, dA, dB, base):
    ids, G = c["ids"].cpu().numpy(), c["A"].shape[0]
    x, dy, A, B, f, t = (wide(c["X"]), wide(c["dY"]), wide(c["A"]), wide(c["B"]), wide(c["scale"]), wide(T))
    rx, ra, rb, rt = adapt.lora_backward(dy, x, t, A, B, ids, f, None if base is None else wide(base))
    fi = _per_row(c, f)
    dt = np.abs(fi)[:, None] * (_links(dy.shape[1]) * _dots(dy, B, ids, G)) + 2 * EPS32 * np.abs(rt)
    if dX is not None:
        parts = 2.0 ** -20 if dX.dtype == F16 else 2.0 ** -15
        near(dX, rx, _add_bound(rt, dt, A, ids, np.ones(len(ids)), parts) + 2 * EPS32 * np.abs(rx), "dX")
    for g in range(G):
        i = np.nonzero(ids == g)[0]
        link = _links(len(i))
        top = np.abs(rt[i]).max(axis=0) if len(i) else np.zeros(rt.shape[1])
        ba = (dt[i] + link * np.abs(rt[i]) + 2.0 ** -20 * top).T @ np.abs(x[i])
        near(dA[g], ra[g], ba, f"dA[{g}]")
        ft = np.abs(f[g] * t[i])
        top = ft.max(axis=0) if len(i) else np.zeros(t.shape[1])
        near(dB[g], rb[g], ((link + 4 * EPS32) * ft + 2.0 ** -20 * top).T @ np.abs(dy[i]), f"dB[{g}]")


SHAPES = [  # s, h, o, r, G, ids
    (1, 64, 64, 1, 1, "one"), (1, 4096, 512, 8, 4, "one"), (2, 64, 192, 3, 2, "mixed"), (7, 320, 64, 16, 3, "none"),
    (15, 128, 256, 17, 3, "odd"), (16, 192, 128, 16, 70, "mixed"), (17, 256, 448, 33, 1, "one"),
    (32, 64, 1024, 128, 2, "mixed"), (33, 1024, 64, 5, 5, "runs"), (64, 2048, 640, 16, 24, "mixed"),
    (65, 512, 576, 64, 2, "odd"), (129, 576, 320, 100, 3, "runs"), (300, 768, 704, 8, 4, "runs"),
    (511, 256, 256, 32, 2, "one"), (700, 320, 192, 12, 9, "mixed"), (1030, 128, 64, 127, 1, "odd"),
    (2100, 64, 128, 4, 300, "mixed"), (260, 4160, 4224, 16, 3, "runs"), (400, 1088, 640, 64, 3, "runs"),
    (330, 320, 2112, 48, 2, "mixed"), (1100, 2048, 1024, 64, 1, "one"), (256, 128, 576, 20, 2, "mixed"),
    (255, 192, 64, 8, 300, "mixed"), (257, 1024, 192, 40, 6, "odd"), (256, 640, 64, 70, 1, "one"),
    (1500, 1024, 4160, 64, 5, "runs"), (2050, 2048, 1088, 96, 4, "mixed"), (1111, 4096, 256, 40, 20, "odd"),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", SHAPES)
def test_forward_and_backward(s, h, o, r, G, kind, dtype):
    say(f"  launch: lora s={s} h={h} o={o} r={r} G={G} {kind} {dtype}")
    c = _case(s, h, o, r, G, kind, dtype)
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    torch.cuda.synchronize()
    _check_forward(c, Y, T, c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])
    torch.cuda.synchronize()
    _check_backward(c, T, dX, dA, dB, c["gbase"])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G", [(5, 128, 192, 9, 2), (90, 384, 256, 24, 3)])
def test_without_base_in_place_and_strided(s, h, o, r, G, dtype):
    c = _case(s, h, o, r, G, "mixed", dtype, seed=1)
    args = (c["A"], c["B"], c["ids"], c["scale"])
    say(f"  launch: lora variants s={s} {dtype}")
    Y, T = i8.lora_forward(c["X"], *args)
    _check_forward(c, Y, T, None)
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, *args)
    _check_backward(c, T, dX, dA, dB, None)
    none, dA1, dB1 = i8.lora_backward(c["dY"], c["X"], T, *args, input_grad=False)
    assert none is None and torch.equal(dA, dA1) and torch.equal(dB, dB1)
    # views of wider buffers, the rest of which holds NaN
    Xs, bs, dYs, gs = (strided(c[k], 8 * (j + 1), 8 * j) for j, k in enumerate(("X", "base", "dY", "gbase")))
    Y0, _ = i8.lora_forward(c["X"], *args, base=c["base"])
    dX0, dA0, dB0 = i8.lora_backward(c["dY"], c["X"], T, *args, base=c["gbase"])
    Y1, T1 = i8.lora_forward(Xs, *args, base=bs, Y=bs)
    dX1, dA1, dB1 = i8.lora_backward(dYs, Xs, T1, *args, base=gs, dX=gs)
    for a, b in ((Y0, Y1), (T, T1), (dX0, dX1), (dA0, dA1), (dB0, dB1)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_no_tokens(dtype):
    c = _case(0, 128, 64, 4, 3, "one", dtype)
    say("  launch: lora with no tokens")
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"])
    torch.cuda.synchronize()
    assert Y.shape == (0, 64) and T.shape == (0, 4) and dX.shape == (0, 128)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,kind", [(40, "mixed"), (200, "runs")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_where_they_belong(s, kind, bad, dtype):
    """A bad row reaches its own row of T, Y and dX and its own adapter's
    gradients; a bad adapter reaches its own rows; nothing else changes a bit."""
    G, r = 4, 20
    c = _case(s, 256, 320, r, G, kind, dtype, seed=2)
    ids = c["ids"].cpu().numpy()
    row = int(np.nonzero(ids == 1)[0][0])
    args = (c["A"], c["B"], c["ids"], c["scale"])

    def everything(c):
        Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
        return (Y, T) + i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])

    say(f"  launch: lora with bad values s={s} {kind} {bad} {dtype}")
    good = everything(c)
    d = dict(c, X=c["X"].clone(), dY=c["dY"].clone())
    d["X"][row, 3] = bad
    d["dY"][row, 5] = bad
    got = everything(d)
    others = torch.from_numpy(np.arange(s) != row)
    for a, b in zip(good[:3], got[:3]):
        assert torch.equal(a[others], b[others])
        assert not torch.isfinite(b[row]).all()
    for a, b in zip(good[3:], got[3:]):
        keep = [g for g in range(G) if g != 1]
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(b[1]).all()
    d = dict(c, A=c["A"].clone(), B=c["B"].clone())
    d["A"][2] = bad
    d["B"][2] = bad
    got = everything(d)
    others = torch.from_numpy(ids != 2)
    for a, b in zip(good[:3], got[:3]):
        assert torch.equal(a[others], b[others])
        assert not torch.isfinite(b[~others]).any()
    # a row that no adapter may touch: garbage in X and dY there changes no gradient
    d = dict(c, X=c["X"].clone(), dY=c["dY"].clone())
    bare = torch.from_numpy((ids < 0) | (ids >= G))
    assert bare.any()
    d["X"][bare] = bad
    d["dY"][bare] = bad
    got = everything(d)
    for a, b in zip(good, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_and_small_factors(dtype):
    """T and dT are fp32: factors beyond fp16's range and far below its
    smallest step keep their digits, also beside each other."""
    c = _case(70, 512, 256, 16, 2, "runs", dtype, seed=3)
    c["X"][:20] *= 2000.0
    c["dY"][10:50] *= 2.0 ** -8
    c["dY"] *= 2.0 ** -3
    c["A"] *= 16.0
    c["B"] *= 2.0 ** -4
    say(f"  launch: lora with wide ranges {dtype}")
    c["base"] = torch.zeros_like(c["base"])
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"] * 2.0 ** -8, base=c["base"])
    d = dict(c, scale=c["scale"] * 2.0 ** -8)
    _check_forward(d, Y, T, c["base"])
    if dtype == F16:
        assert float(T.abs().max()) > 65504
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"])
    _check_backward(c, T, dX, dA, dB, None)


def test_same_bits_on_every_call_other_streams_and_replays():
    c = _case(300, 1024, 2048, 16, 3, "mixed", F16, seed=4)
    args = (c["A"], c["B"], c["ids"], c["scale"])
    Y0, T0 = i8.lora_forward(c["X"], *args, base=c["base"])
    ref = i8.lora_backward(c["dY"], c["X"], T0, *args, base=c["gbase"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("  launch: lora on a second stream")
    with torch.cuda.stream(side):
        Y1, T1 = i8.lora_forward(c["X"], *args, base=c["base"])
        got = i8.lora_backward(c["dY"], c["X"], T1, *args, base=c["gbase"])
    torch.cuda.synchronize()
    for a, b in zip((Y0, T0) + ref, (Y1, T1) + got):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    say("  capture: lora forward and backward")
    with torch.cuda.graph(g):
        Y2, T2 = i8.lora_forward(c["X"], *args, base=c["base"])
        got = i8.lora_backward(c["dY"], c["X"], T2, *args, base=c["gbase"])
    for k in range(3):
        for t in (Y2, T2) + got:
            t.fill_(float("nan"))
        i8.lora_forward(c["X"], *args)
        torch.cuda.synchronize()
        say(f"  replay {k + 1}")
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((Y0, T0) + ref, (Y2, T2) + got):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """The slope of <dY, lora_forward> along a direction, by central
    differences of the definition in 64 bits, against the kernels' gradients.
    X, A and B are multiples of 2^-6 below 4 in magnitude, so fp16 holds them
    exactly; the function is of third degree, and a step of 1e-3 is off by
    1e-6 of the direction's cubic term. dX carries fp16's rounding, 2^-11 of
    each value; random signs leave less of it in the sum, and 2^-11 of the
    norms bounds it. dA and dB are fp32: 1e-5."""
    rng = np.random.default_rng(9)
    s, h, o, r, G = 24, 64, 128, 4, 2
    grid = lambda shape: torch.from_numpy(np.round(rng.normal(size=shape) * 20).clip(-255, 255).astype(np.float32)   # noqa: E731
                                          / 64).to(DEV).half()
    X, A, B, dY = grid((s, h)), grid((G, r, h)), grid((G, r, o)), grid((s, o))
    ids = _ids(rng, s, G, "mixed")
    scale = torch.tensor([0.5, 2.0], device=DEV)
    _, T = i8.lora_forward(X, A, B, ids, scale)
    grads = i8.lora_backward(dY, X, T, A, B, ids, scale)
    at = [wide(X), wide(A), wide(B)]
    for k, tol in ((0, 2.0 ** -11), (1, 1e-5), (2, 1e-5)):
        v = rng.normal(size=at[k].shape)
        f = [np.sum(wide(dY) * adapt.lora_forward(*[a + t * v if j == k else a for j, a in enumerate(at)],
                                                  ids.cpu().numpy(), wide(scale), None)[0]) for t in (1e-3, -1e-3)]
        g = wide(grads[k])
        assert abs((f[0] - f[1]) / 2e-3 - np.sum(g * v)) <= tol * np.linalg.norm(g) * np.linalg.norm(v)


def test_rows_and_adapters_beyond_32_bit_offsets():
    """Y with more than 2^31 elements, and adapters with more than 2^31."""
    s, h, o, r, G = 2 ** 15 + 3, 64, 65600, 2, 2
    say(f"  launch: lora s={s} o={o}")
    rng = np.random.default_rng(6)
    X, A, B = randn(rng, (s, h), F16), randn(rng, (G, r, h), F16, 0.1), randn(rng, (G, r, o), F16, 0.1)
    ids = torch.zeros(s, dtype=torch.int32, device=DEV)
    ids[-9:] = 1
    scale = torch.ones(G, device=DEV)
    Y, T = i8.lora_forward(X, A, B, ids, scale)
    c = dict(X=X[-20:], A=A, B=B, ids=ids[-20:], scale=scale)
    _check_forward(c, Y[-20:], T[-20:], None)
    del Y
    G, r, h, o = 300, 128, 64 * 1000, 64
    say(f"  launch: lora G={G} h={h}")
    A = torch.zeros((G, r, h), dtype=F16, device=DEV)
    A[-1] = randn(rng, (r, h), F16, 0.1)
    B = randn(rng, (G, r, o), F16, 0.1)
    X = randn(rng, (3, h), F16)
    ids = torch.tensor([G - 1, 0, G - 1], dtype=torch.int32, device=DEV)
    Y, T = i8.lora_forward(X, A, B, ids, torch.ones(G, device=DEV))
    near(T[::2], wide(X[::2]) @ wide(A[-1]).T, _links(h) * (np.abs(wide(X[::2])) @ np.abs(wide(A[-1])).T), "T")
    assert not T[1].any()


def test_refusals():
    c = _case(4, 128, 64, 4, 2, "one", F16)
    X, A, B, ids, f = (c[k] for k in ("X", "A", "B", "ids", "scale"))
    T = torch.zeros((4, 4), device=DEV)
    for call in (lambda: i8.lora_forward(X.float(), A, B, ids, f), lambda: i8.lora_forward(X, A.to(BF16), B, ids, f),
                 lambda: i8.lora_forward(X, A, B, ids.long(), f), lambda: i8.lora_forward(X, A, B, ids[:3], f),
                 lambda: i8.lora_forward(X, A, B, ids, f[:1]), lambda: i8.lora_forward(X, A[0], B, ids, f),
                 lambda: i8.lora_forward(X, A, B[:1], ids, f), lambda: i8.lora_forward(X, A[:, :, :64], B, ids, f),
                 lambda: i8.lora_forward(X.cpu(), A, B, ids, f), lambda: i8.lora_forward(X, A, B, ids, f, base=X),
                 lambda: i8.lora_forward(X, A, B, ids.cpu(), f), lambda: i8.lora_forward(X, A, B, ids, f, T=T[:, :3]),
                 lambda: i8.lora_backward(X, X, T, A, B, ids, f),
                 lambda: i8.lora_backward(c["dY"], X, T.half(), A, B, ids, f),
                 lambda: i8.lora_forward(X, A, B, ids, f, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros(4 * 136 + 4, dtype=F16, device=DEV)
    for call in (lambda: i8.lora_forward(odd[4:4 + 4 * 128].view(4, 128), A, B, ids, f),                 # alignment
                 lambda: i8.lora_forward(odd[:4 * 132].view(4, 132)[:, :128], A, B, ids, f),             # row stride
                 lambda: i8.lora_forward(X[:, :96].contiguous(), A[:, :, :96].contiguous(), B, ids, f),  # h % 64
                 lambda: i8.lora_forward(X, torch.zeros((2, 129, 128), dtype=F16, device=DEV),
                                         torch.zeros((2, 129, 64), dtype=F16, device=DEV), ids, f),      # rank
                 lambda: i8.lora_backward(c["dY"], X, T, A, B, ids, f, dX=X)):                           # overlap
        with pytest.raises(i8.I8MMError):
            call()
