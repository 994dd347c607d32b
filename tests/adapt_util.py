"""Helpers of the GPU tests of layer norm, the adapters and clipping: inputs of
the three element types, their values in 64 bits, and bounds."""

from __future__ import annotations

import numpy as np
import torch

from gpu_util import DEV

EPS32 = 2.0 ** -24                       # half an ulp of 1 in fp32
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}
# half a step of the subnormal numbers, below which a type holds nothing
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def randn(rng: np.random.Generator, shape, dtype: torch.dtype, std: float = 1.0) -> torch.Tensor:
    return torch.from_numpy(np.asarray(rng.normal(size=shape) * std, np.float32)).to(DEV).to(dtype)


def wide(t: torch.Tensor) -> np.ndarray:
    """The values of a tensor in 64 bits."""
    return t.detach().double().cpu().numpy()


def strided(t: torch.Tensor, extra: int, offset: int = 0) -> torch.Tensor:
    """A copy of a matrix as a view with `extra` more elements a row (filled
    with NaN), starting `offset` elements into its storage."""
    s, h = t.shape
    store = torch.full((offset + s * (h + extra) + 8,), float("nan"), dtype=t.dtype, device=t.device)
    view = store[offset:offset + s * (h + extra)].view(s, h + extra)[:, :h]
    view.copy_(t)
    return view


def near(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str) -> None:
    """|got - ref| <= bound + half an ulp of got's type, element by element."""
    g = wide(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    if g.size == 0:
        return
    limit = bound + HALF_ULP[got.dtype] * (np.abs(ref) + bound) + SMALLEST[got.dtype]
    off = np.abs(g - ref)
    bad = ~(off <= limit)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound, first at {at}: "
                             f"{g[at]!r} for {ref[at]!r}, bound {np.broadcast_to(limit, g.shape)[at]:.3e}")
