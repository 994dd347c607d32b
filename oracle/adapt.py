"""Layer norm, low-rank adapters and gradient clipping in 64 bits, from their
definitions (numpy, CPU). Test infrastructure: shares no code with the GPU
path. Every argument is converted to float64 first.
"""

from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

F = np.float64


def layer_norm(X, weight, bias, eps) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(Y, mean, rstd) of the rows of X."""
    X = np.asarray(X, F)
    mean = X.mean(axis=1)
    d = X - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    Y = d * rstd[:, None] * np.asarray(weight, F)
    return (Y if bias is None else Y + np.asarray(bias, F)), mean, rstd


def layer_norm_backward(dY, X, weight, mean, rstd) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(dX, d_weight, d_bias) for the gradient dY, given the rows' statistics."""
    dY, X, rstd = np.asarray(dY, F), np.asarray(X, F), np.asarray(rstd, F)[:, None]
    n = (X - np.asarray(mean, F)[:, None]) * rstd
    g = dY * np.asarray(weight, F)
    mean_g = g.mean(axis=1, keepdims=True)
    mean_gn = (g * n).mean(axis=1, keepdims=True)
    return rstd * (g - mean_g - n * mean_gn), (dY * n).sum(axis=0), dY.sum(axis=0)


def _groups(ids, G):
    ids = np.asarray(ids)
    return [(g, np.nonzero(ids == g)[0]) for g in range(G) if (ids == g).any()]


def lora_forward(X, A, B, ids, scale, base: Optional[np.ndarray]) -> Tuple[np.ndarray, np.ndarray]:
    """(Y, T): Y_i = base_i + scale_g T_i B_g with T_i = X_i A_g^T, g = ids[i]."""
    X, A, B = np.asarray(X, F), np.asarray(A, F), np.asarray(B, F)
    T = np.zeros((X.shape[0], A.shape[1]))
    Y = np.zeros((X.shape[0], B.shape[2])) if base is None else np.array(base, F)
    for g, i in _groups(ids, A.shape[0]):
        T[i] = X[i] @ A[g].T
        Y[i] = Y[i] + F(scale[g]) * (T[i] @ B[g])
    return Y, T


def lora_backward(dY, X, T, A, B, ids, scale, base: Optional[np.ndarray]
                  ) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """(dX, dA, dB, dT) of lora_forward for the gradient dY, given T."""
    dY, X, T, A, B = (np.asarray(v, F) for v in (dY, X, T, A, B))
    dX = np.zeros_like(X) if base is None else np.array(base, F)
    dA, dB, dT = np.zeros_like(A), np.zeros_like(B), np.zeros_like(T)
    for g, i in _groups(ids, A.shape[0]):
        dT[i] = F(scale[g]) * (dY[i] @ B[g].T)
        dX[i] = dX[i] + dT[i] @ A[g]
        dA[g] = dT[i].T @ X[i]
        dB[g] = F(scale[g]) * (T[i].T @ dY[i])
    return dX, dA, dB, dT


def clip_grad_norm(grads: Sequence[np.ndarray], max_norm: float) -> Tuple[float, List[np.ndarray]]:
    """(N, the gradients times min(1, max_norm / (N + 1e-6))); the factor is 1
    if max_norm is infinite, whatever N is but NaN."""
    grads = [np.asarray(g, F) for g in grads]
    total = np.sqrt(sum(float(np.sum(g * g)) for g in grads))
    c = total if np.isnan(total) else 1.0 if np.isinf(max_norm) else min(1.0, max_norm / (total + 1e-6))
    with np.errstate(invalid="ignore"):          # 0 times an infinity
        return float(total), [c * g for g in grads]
