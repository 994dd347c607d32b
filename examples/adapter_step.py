"""One training step of an adapted int8 layer, and one decoding step of it.

The layer is  norm -> frozen int8 projection -> + low-rank adapters.  Training
changes the adapters and the norm's parameters; the projection's weights stay
int8, and its own part of the input's gradient is the library's dense product
with the transposed weights, packed once at load time.

    python examples/adapter_step.py [--steps 5]

needs a gfx950 GPU and the built library.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_quantized_matmul_amd as i8  # noqa: E402


class AdaptedLayer:
    """norm -> int8 projection + adapters, [h] -> [o] features."""

    def __init__(self, W: torch.Tensor, n_adapters: int, rank: int, alpha: float, seed: int = 0):
        dev, (h, o) = W.device, W.shape
        g = torch.Generator(device=dev).manual_seed(seed)
        self.W = W                                                  # fp16 [h, o], for the outlier columns
        self.Wq, self.c_w = i8.quantize_colwise_weights(W)          # the frozen projection
        self.Wt = i8.pack_fp16_weights(W.t().contiguous())          # for its input's gradient
        self.norm_weight = torch.ones(h, dtype=torch.float32, device=dev)
        self.norm_bias = torch.zeros(h, dtype=torch.float32, device=dev)
        self.A = (torch.randn((n_adapters, rank, h), generator=g, device=dev) / h ** 0.5).half()
        self.B = torch.zeros((n_adapters, rank, o), dtype=torch.float16, device=dev)   # starts as the base model
        self.scale = torch.full((n_adapters,), alpha / rank, dtype=torch.float32, device=dev)

    def forward(self, X: torch.Tensor, ids: torch.Tensor):
        """X fp16 [s, h], ids int32 [s] (the adapter of each row, -1: none) -> (Y, what backward needs)."""
        N, mean, rstd = i8.layer_norm(X, self.norm_weight, self.norm_bias)
        C = i8.forward(N, self.Wq, self.c_w, self.W)
        Y, T = i8.lora_forward(N, self.A, self.B, ids, self.scale, base=C, Y=C)
        return Y, (X, N, mean, rstd, T, ids)

    def backward(self, dY: torch.Tensor, saved):
        """-> (dX, gradients of [A, B, norm_weight, norm_bias] in fp32)."""
        X, N, mean, rstd, T, ids = saved
        dN = i8.fp16_gemm(dY, self.Wt)                              # through the frozen projection
        dN, dA, dB = i8.lora_backward(dY, N, T, self.A, self.B, ids, self.scale, base=dN, dX=dN)
        dX, d_weight, d_bias = i8.layer_norm_backward(dN, X, self.norm_weight, mean, rstd)
        return dX, [dA, dB, d_weight, d_bias]

    def step(self, grads, lr: float, max_norm: float) -> torch.Tensor:
        """Clips the gradients and takes a plain gradient step; -> their norm before clipping."""
        total = i8.clip_grad_norm(grads, max_norm)
        for p, g in zip((self.A, self.B, self.norm_weight, self.norm_bias), grads):
            p -= (lr * g).to(p.dtype)
        return total


def train(layer: AdaptedLayer, X, ids, target, steps: int, lr: float = 4.0, max_norm: float = 1.0):
    """Mean squared error to `target` over rows with an adapter; -> the losses."""
    losses = []
    rows = (ids >= 0)[:, None]
    for _ in range(steps):
        Y, saved = layer.forward(X, ids)
        diff = torch.where(rows, Y.float() - target, 0.0)
        losses.append(float(diff.square().mean()))
        dY = (diff * (2.0 / diff.numel()) * 2.0 ** 12).half()       # loss scale of 2^12
        _, grads = layer.backward(dY, saved)
        for g in grads:
            g *= 2.0 ** -12
        layer.step(grads, lr, max_norm)
    return losses


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    s, h, o = 512, 1024, 2048
    W = (0.02 * torch.randn((h, o), generator=g, device="cuda")).half()
    layer = AdaptedLayer(W, n_adapters=3, rank=8, alpha=16.0)
    X = torch.randn((s, h), generator=g, device="cuda").half()
    ids = torch.arange(s, device="cuda").div(s // 4, rounding_mode="floor").int() - 1   # the first quarter: none
    target = torch.randn((s, o), generator=g, device="cuda")
    for k, loss in enumerate(train(layer, X, ids, target, a.steps)):
        print(f"step {k}: loss {loss:.5f}")
    Y, _ = layer.forward(X[:3], torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda"))
    print(f"decoded 3 tokens with adapters 0, none, 2: {tuple(Y.shape)}, finite: {bool(torch.isfinite(Y).all())}")


if __name__ == "__main__":
    main()
