"""Helpers of the GPU tests of decoding: paged caches with NaN wherever no
sequence's tokens are, and the bounds of the attention over them."""

from __future__ import annotations

import numpy as np
import torch

from adapt_util import HALF_ULP, wide
from gpu_util import DEV

I32 = torch.int32


def ints(a) -> torch.Tensor:
    return torch.as_tensor(np.asarray(a, np.int32), device=DEV)


def paged(rng, lens, page, spare=3, width=None):
    """(tables [n, width], pages): each sequence's pages, in no order; unused entries are -1."""
    need = [-(-max(0, n) // page) for n in lens]
    width = max(need + [1]) if width is None else width
    ids = list(rng.permutation(sum(need) + spare))
    tables = np.full((len(lens), width), -1, np.int32)
    for i, k in enumerate(need):
        for c in range(k):
            tables[i, c] = ids.pop()
    return tables, sum(need) + spare


def pool(rng, tables, lens, pages, heads, page, d, dtype, gap=0, std=1.0):
    """[pages, heads, page, d] of `dtype` with `gap` elements between pages: N(0, std) where a sequence's
    tokens are, NaN elsewhere."""
    store = torch.full((pages, heads * page * d + gap), float("nan"), dtype=dtype, device=DEV)
    out = store[:, :heads * page * d].view(pages, heads, page, d)
    for i, n in enumerate(lens):
        for c in range(-(-max(0, n) // page)):
            if not 0 <= tables[i, c] < pages:
                continue
            m = min(page, n - c * page)
            v = np.asarray(rng.normal(size=(heads, m, d)) * std, np.float32)
            out[int(tables[i, c]), :, :m] = torch.from_numpy(v).to(DEV).to(dtype)
    return out


def attention_bounds(q, K_pages, V_pages, tables, lens, scale, slopes, dtype):
    """(bound of out, bound of lse) around the 64-bit result, before out's own rounding.

    With s in powers of 2, an fp32 chain of d products and sums gives s off by (d + 4) 2^-24 sum |q k| scale log2 e,
    the factor, the bias and their sum by 2^-22 |s| and 2^-22 |slope t|; 2^s is off by that times ln 2 and by 2^-22. A
    probability is rounded to the cache's type (half a step, or 2^-40 of the largest where it is subnormal there).
    The sums are chains of at most len / 16 + 80 additions in fp32, each partial sum at most sum |terms|."""
    q, Kp, Vp = wide(q), wide(K_pages), wide(V_pages)
    P, kv, page, d = Kp.shape
    n, M = tables.shape
    heads = q.shape[1] // d
    u = HALF_ULP[dtype]
    bo, bl = np.zeros((n, heads, d)), np.zeros((n, heads))
    for i in range(n):
        length = min(max(int(lens[i]), 0), M * page)
        at = np.array([t for t in range(length) if 0 <= tables[i, t // page] < P], int)
        if not len(at):
            continue
        ids = tables[i, at // page]
        k, v = Kp[ids, :, at % page], Vp[ids, :, at % page]
        row = q[i].reshape(heads, d)
        for a in range(heads):
            kk, vv = k[:, a // (heads // kv)], v[:, a // (heads // kv)]
            bias = 0.0 if slopes is None else float(slopes[a]) * (at - (length - 1))
            s = scale * (kk @ row[a]) + bias
            off = (d + 4) * 2.0 ** -24 * abs(scale) * (np.abs(kk) @ np.abs(row[a])) + 2.0 ** -22 * (np.abs(s) + np.abs(bias))
            off = off * 1.5 + 2.0 ** -22 + 2.0 ** -22 * np.abs(s - s.max())
            w = np.exp(s - s.max())
            total = w.sum()
            chain = (len(at) / 16 + 80) * 2.0 ** -24
            part = ((u + off + chain) * w + 2.0 ** -40) / total
            drift = (off * w).sum() / total + chain
            bo[i, a] = part @ np.abs(vv) + drift * ((w / total) @ np.abs(vv))
            lse = s.max() + np.log(total)
            bl[i, a] = drift + off[s.argmax()] + 2.0 ** -22 * abs(lse) + 2.0 ** -20
    return bo.reshape(n, heads * d), bl
