"""The adapters' gradients for so many adapters that their blocks do not fit
one launch: a dimension of a grid has fewer than 2^32 threads."""

import pytest
import torch

import int8_quantized_matmul_amd as i8
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

G, H, O = 65535, 64, 32832               # (H + O) / 128 blocks of 256 threads for each adapter: more than 2^32


def _inputs(s, ids):
    g = torch.Generator(device=DEV).manual_seed(2)
    make = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)   # noqa: E731
    c = dict(X=make(s, H), dY=make(s, O), A=make(G, 1, H), B=make(G, 1, O), ids=ids.to(torch.int32))
    c["scale"] = 0.5 + torch.rand(G, generator=g, device=DEV)
    return c


def _run(c, s):
    T = torch.linspace(1, 2, s, device=DEV)[:, None].contiguous()
    dA, dB = (torch.full((G, 1, n), float("nan"), device=DEV) for n in (H, O))
    say(f"  launch: lora_backward s={s} G={G} o={O}")
    i8.lora_backward(c["dY"], c["X"], T, c["A"], c["B"], c["ids"], c["scale"], input_grad=False, dA=dA, dB=dB)
    torch.cuda.synchronize()
    return T, dA, dB


def _same(c, T, dA, dB, tokens):
    """One token for each of its adapters: no sums but dT's, whose bound is 2^-10 of its terms' root of squares."""
    for i0 in range(0, len(tokens), 4096):
        i = tokens[i0:i0 + 4096]
        g = c["ids"][i].long()
        f, dy = c["scale"][g][:, None], c["dY"][i].float()
        want = f * T[i] * dy
        assert bool(((dB[g, 0] - want).abs() <= 2.0 ** -20 * want.abs()).all())
        B = c["B"][g, 0].float()
        dt = f * (dy.double() * B.double()).sum(1, keepdim=True).float()
        off = f * 2.0 ** -10 * (dy * B).square().sum(1, keepdim=True).sqrt() + 2.0 ** -20 * dt.abs()
        x = c["X"][i].float()
        assert bool(((dA[g, 0] - dt * x).abs() <= off * x.abs()).all())


def test_zeros_of_adapters_that_no_token_carries():
    s = 60
    ids = torch.full((s,), -1, device=DEV)
    tokens = torch.arange(0, s, 3, device=DEV)
    ids[tokens] = G - 1 - 3276 * torch.arange(20, device=DEV)
    c = _inputs(s, ids)
    T, dA, dB = _run(c, s)
    _same(c, T, dA, dB, tokens)
    for d in (dA, dB):
        some = torch.cat([d[k:k + 4096].abs().sum((1, 2)) for k in range(0, G, 4096)])
        assert bool((some.nonzero().flatten() == ids[tokens].sort().values).all()) and not torch.isnan(some).any()


def test_an_adapter_for_each_token():
    ids = torch.randperm(G, generator=torch.Generator().manual_seed(3)).to(DEV)
    c = _inputs(G, ids)
    T, dA, dB = _run(c, G)
    _same(c, T, dA, dB, torch.arange(G, device=DEV))
