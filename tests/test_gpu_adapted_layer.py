"""The new operators together, as examples/adapter_step.py uses them: its
layer's forward and backward pass against the same composition in 64 bits
around the projection's own output, and its training step lowers the loss.

Bounds: N is rounded to fp16 (2^-11), so is the projection's output, to which
the adapters add; what follows from N's rounding is left out by comparing with
the definitions applied to the layer's own N. Y: half an ulp of fp16 and 2^-19
of the terms. The gradients that reach the norm are fp16 twice (the projection's
part and the sum): 2^-10 of their size, relative to the largest of a row.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

import int8_quantized_matmul_amd as i8
from adapt_util import near, wide
from gpu_util import DEV, say
from oracle import adapt

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("adapter_step", os.path.join(ROOT, "examples", "adapter_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _layer(m, h, o):
    g = torch.Generator(device=DEV).manual_seed(3)
    layer = m.AdaptedLayer((0.02 * torch.randn((h, o), generator=g, device=DEV)).half(), 3, 8, 16.0)
    layer.B = (0.05 * torch.randn(layer.B.shape, generator=g, device=DEV)).half()
    return layer, g


def test_forward_and_backward_against_the_definitions():
    m = _example()
    s, h, o = 300, 512, 768
    layer, g = _layer(m, h, o)
    X = torch.randn((s, h), generator=g, device=DEV).half()
    ids = (torch.arange(s, device=DEV) % 4).int() - 1
    say("  launch: adapted layer forward and backward")
    Y, saved = layer.forward(X, ids)
    N, T = saved[1], saved[4]
    C = i8.forward(N, layer.Wq, layer.c_w, layer.W)
    A, B, f, k = wide(layer.A), wide(layer.B), wide(layer.scale), ids.cpu().numpy()
    ry, rt = adapt.lora_forward(wide(N), A, B, k, f, wide(C))
    near(Y, ry, 2.0 ** -19 * (np.abs(ry) + np.abs(f[0]) * (np.abs(rt) @ np.abs(B).max(axis=0))), "Y")
    dY = (1e-2 * torch.randn((s, o), generator=g, device=DEV)).half()
    dX, grads = layer.backward(dY, saved)
    torch.cuda.synchronize()
    dn = wide(dY) @ wide(layer.W).T
    dn, ra, rb, _ = adapt.lora_backward(wide(dY), wide(N), wide(T), A, B, k, f, dn)
    rx, rw, rbias = adapt.layer_norm_backward(dn, wide(X), wide(layer.norm_weight), wide(saved[2]), wide(saved[3]))
    off = 2.0 ** -10 * np.abs(dn).max()
    near(dX, rx, 4 * off * wide(saved[3]).max() * np.ones_like(rx), "dX")
    near(grads[0], ra, 1e-4 * np.abs(ra).max() * np.ones_like(ra), "dA")
    near(grads[1], rb, 1e-4 * np.abs(rb).max() * np.ones_like(rb), "dB")
    n = (wide(X) - wide(saved[2])[:, None]) * wide(saved[3])[:, None]
    near(grads[2], rw, off * np.abs(n).sum(axis=0), "d_weight")
    near(grads[3], rbias, off * s * np.ones(h), "d_bias")


def test_training_lowers_the_loss_and_decoding_agrees():
    m = _example()
    layer, g = _layer(m, 256, 512)
    X = torch.randn((400, 256), generator=g, device=DEV).half()
    ids = (torch.arange(400, device=DEV) // 100).int() - 1
    target = torch.randn((400, 512), generator=g, device=DEV)
    say("  launch: adapted layer training steps")
    losses = m.train(layer, X, ids, target, 8)
    assert losses[-1] < losses[0] and all(np.isfinite(losses))
    # the same rows one at a time: the adapters' few-token form against the many-token one
    Y, saved = layer.forward(X, ids)
    N = saved[1]
    C = i8.forward(N, layer.Wq, layer.c_w, layer.W)
    args = (layer.A, layer.B)
    all_rows, T = i8.lora_forward(N, *args, ids, layer.scale, base=C)
    for i in (0, 99, 100, 399):
        one, t = i8.lora_forward(N[i:i + 1], *args, ids[i:i + 1], layer.scale, base=C[i:i + 1])
        assert torch.allclose(t, T[i:i + 1], rtol=1e-5, atol=1e-5)
        assert torch.allclose(one.float(), all_rows[i:i + 1].float(), rtol=2.0 ** -10, atol=2.0 ** -10)
