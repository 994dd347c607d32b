"""The adapters' gradients where ranks differ: in size, and in being finite.

The bounds are test_gpu_lora.py's, which group a rank's factors with that
rank's own tokens alone: a rank's gradient depends on no other rank.
"""

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, wide
from gpu_util import say
from oracle import adapt
from test_gpu_lora import BF16, F16, _case, _check_backward, _links

pytestmark = pytest.mark.gpu

# s, h, o, r, G, ids: one launch with partial sums, one without; ranks in one tile, in several, shared by wavefronts
CASES = [(40, 128, 192, 5, 2, "runs"), (300, 256, 320, 20, 2, "mixed"), (700, 320, 256, 40, 1, "one"),
         (600, 192, 128, 100, 3, "runs")]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("s,h,o,r,G,kind", CASES)
def test_ranks_far_apart_in_size(s, h, o, r, G, kind, dtype):
    """Every second rank of A and B is 2^-29 of its neighbours'. Both are
    multiples of 2^-24, so that fp16 holds them exactly."""
    c = _case(s, h, o, r, G, kind, dtype, seed=5)
    for k in ("A", "B"):
        small = (torch.randint(-15, 16, c[k].shape, device=c[k].device) * 2.0 ** -24).to(dtype)
        c[k] = (c[k] * 2.0 ** 9).to(dtype)
        c[k][:, 1::2] = small[:, 1::2]
    say(f"  launch: lora ranks far apart s={s} r={r} {kind} {dtype}")
    _, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"], base=c["base"])
    dX, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], base=c["gbase"])
    torch.cuda.synchronize()
    _check_backward(c, T, dX, dA, dB, c["gbase"])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("s,h,o,r,G,kind", CASES)
def test_a_rank_that_is_not_finite_leaves_the_others(s, h, o, r, G, kind, bad, dtype):
    """One rank of adapter 0 is not finite, in A and in B; T is beyond fp16's
    range in some tokens. The other ranks' gradients are the definition's."""
    c = _case(s, h, o, r, G, kind, dtype, seed=6)
    c["X"][::3] *= 2000.0
    c["A"] *= 100.0
    c["dY"] *= 2.0 ** -6
    for k in ("A", "B"):
        c[k][0, r // 2] = bad
    say(f"  launch: lora with a bad rank s={s} r={r} {kind} {bad} {dtype}")
    _, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"])
    _, dA, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], input_grad=False)
    torch.cuda.synchronize()
    ids, f = c["ids"].cpu().numpy(), wide(c["scale"])
    i, keep = np.nonzero(ids == 0)[0], np.arange(r) != r // 2
    assert len(i) and not torch.isfinite(T[i][:, r // 2]).any()
    x, dy, B, t = wide(c["X"])[i], wide(c["dY"])[i], wide(c["B"])[0][keep], wide(T)[i][:, keep]
    zero = np.zeros(len(i), np.int64)
    _, ra, rb, rt = adapt.lora_backward(dy, x, t, np.zeros((1, keep.sum(), h)), B[None], zero, f[:1], None)
    if dtype == F16:
        assert np.abs(t).max() > 65504
    link = _links(len(i))
    dt = f[0] * _links(o) * (np.abs(dy) @ np.abs(B).T) + 2.0 ** -23 * np.abs(rt)
    ba = (dt + link * np.abs(rt) + 2.0 ** -20 * np.abs(rt).max(axis=0)).T @ np.abs(x)
    near(dA[0][torch.from_numpy(keep)], ra[0], ba, "dA of the finite ranks")
    ft = np.abs(f[0] * t)
    bb = ((link + 2.0 ** -22) * ft + 2.0 ** -20 * ft.max(axis=0)).T @ np.abs(dy)
    near(dB[0][torch.from_numpy(keep)], rb[0], bb, "dB of the finite ranks")
    assert not torch.isfinite(dA[0, r // 2]).all() and not torch.isfinite(dB[0, r // 2]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_factors_at_the_end_of_fp32(dtype):
    """T between bf16's largest number and fp32's, in dB and, from a product
    that is as large, in Y."""
    c = _case(40, 128, 192, 4, 1, "one", dtype, seed=10)
    top = float(np.finfo(np.float32).max)
    c["scale"].fill_(1.0)
    T = torch.randn((40, 4), generator=torch.Generator().manual_seed(1)).to(c["X"].device)
    T[7, 1], T[9, 2] = top, -0.999 * top
    c["dY"] = (c["dY"] * 2.0 ** -4).to(dtype)
    say(f"  launch: lora with factors at the end of fp32 {dtype}")
    _, _, dB = i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"])
    t, dy = wide(T), wide(c["dY"])
    near(dB[0], t.T @ dy, ((_links(40) + 2.0 ** -20) * np.abs(t)).T @ np.abs(dy) + 2.0 ** -20 * np.abs(t).max(axis=0)[:, None]
         * np.abs(dy).sum(axis=0), "dB")
    if dtype == F16:
        return
    # X A = 255/256 2^128 from two factors of 2^64 and less, B small enough for Y
    c["X"].zero_(), c["A"].zero_(), c["base"].zero_()
    c["X"][:, 3], c["A"][0, :, 3] = 2.0 ** 64, 255 / 256 * 2.0 ** 64
    c["X"][:, 4], c["A"][0, :, 4] = 2.0 ** 56, 0.75 * 2.0 ** 64
    c["B"] = (c["B"] * 2.0 ** -120).to(dtype)
    Y, T = i8.lora_forward(c["X"], c["A"], c["B"], c["ids"], c["scale"])
    t, B = wide(T), wide(c["B"])[0]
    assert np.isfinite(t).all() and np.abs(t).max() > 255.5 * 2.0 ** 120
    near(Y, t @ B, 2.0 ** -14 * (np.abs(t) @ np.abs(B)), "Y")
