"""Decoding between int8 layers from the definitions (numpy, CPU): a paged
key-value cache, the attention of new tokens over it in 64 bits, and beam
search. Test infrastructure: shares no code with the GPU path.
"""

from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

F = np.float64


def append(K, V, K_pages, V_pages, tables, pos, seq=None) -> None:
    """Rows into their slots, in place; rows without one are left out."""
    P, heads, page, d = K_pages.shape
    n, M = tables.shape
    for i in range(len(pos)):
        q, t = i if seq is None else int(seq[i]), int(pos[i])
        if not (0 <= q < n and 0 <= t < M * page):
            continue
        p = int(tables[q, t // page])
        if 0 <= p < P:
            K_pages[p, :, t % page] = K[i].reshape(heads, d)
            V_pages[p, :, t % page] = V[i].reshape(heads, d)


def attention(Q, K_pages, V_pages, tables, lens, scale, slopes=None) -> Tuple[np.ndarray, np.ndarray]:
    """(out [n, heads d], lse [n, heads]) in 64 bits; positions without a page are left out."""
    P, kv, page, d = K_pages.shape
    n, M = tables.shape
    heads = Q.shape[1] // d
    out, lse = np.zeros((n, heads, d)), np.full((n, heads), -np.inf)
    for i in range(n):
        length = min(max(int(lens[i]), 0), M * page)
        at = [t for t in range(length) if 0 <= tables[i, t // page] < P]
        if not at:
            continue
        ids, slots = np.array([tables[i, t // page] for t in at]), np.array([t % page for t in at])
        k, v = (np.asarray(p[ids, :, slots], F) for p in (K_pages, V_pages))       # [tokens, kv, d]
        q = np.asarray(Q[i], F).reshape(heads, d)
        for a in range(heads):
            s = scale * (k[:, a // (heads // kv)] @ q[a])
            if slopes is not None:
                s = s + F(slopes[a]) * (np.array(at) - (length - 1))
            m = s.max()
            with np.errstate(invalid="ignore"):
                w = np.exp(s - m)
                lse[i, a] = m if np.isinf(m) else m + np.log(w.sum())
                out[i, a] = (w / w.sum()) @ v[:, a // (heads // kv)]
    return out.reshape(n, heads * d), lse


def _rows(tables, lens, page) -> Tuple[List[List[int]], List[int]]:
    M = tables.shape[1]
    sizes = [min(max(int(x), 0), M * page) for x in lens]
    return [[int(p) for p in row[:-(-n // page)]] for row, n in zip(tables, sizes)], sizes


def fork(tables, lens, refs, page, parents=None, grow=None, pools: Sequence[np.ndarray] = ()):
    """(tables, lens, refs, state); copied pages are written into the pools."""
    P, M = len(refs), tables.shape[1]
    n = len(lens)
    if parents is None:
        parents = range(n if grow is None else len(grow))
    rows, sizes = _rows(tables, lens, page)
    new = [list(rows[p]) if 0 <= p < n else [] for p in parents]
    size = [sizes[p] if 0 <= p < n else 0 for p in parents]
    refs = [int(r) for r in refs]
    for change, lists in ((-1, rows), (1, new)):
        for row in lists:
            for p in row:
                if 0 <= p < P:
                    refs[p] += change
    grow = [0] * len(new) if grow is None else [max(0, int(g)) for g in grow]
    free = [p for p in range(P) if refs[p] <= 0]
    written = [row[-1] if g and t + g <= M * page and t % page and 0 <= row[-1] < P else None
               for row, t, g in zip(new, size, grow)]
    after, wanted, taken, copied, missed, uncopied = list(refs), 0, 0, [], 0, set()
    for j, (row, t, g) in enumerate(zip(new, size, grow)):
        w = written[j]
        keep = w is not None and w not in written[j + 1:] and written.count(w) >= refs[w]
        copy = w is not None and not keep
        if t + g > M * page:
            missed += 1
            continue
        need = -(-(t + g) // page) - len(row) + copy
        wanted += need
        if (need and wanted > len(free)) or (keep and w in uncopied):
            missed += 1
            if copy:
                uncopied.add(w)
            continue
        got = free[taken:taken + need]
        taken += need
        for p in got:
            after[p] = 1
        if copy:
            copied.append((w, got[0]))
            after[w] -= 1
            row[-1] = got.pop(0)
        row.extend(got)
        size[j] = t + g
    for pool in pools:
        for a, b in copied:
            pool[b] = pool[a]
    out = np.full((len(new), M), -1, np.int32)
    for j, row in enumerate(new):
        out[j, :len(row)] = row
    state = [len(free) - taken, max(0, wanted - len(free)), missed, len(copied)]
    return out, np.array(size, np.int32), np.array(after, np.int32), np.array(state, np.int32)


def compact(tables, refs, pools: Sequence[np.ndarray] = ()):
    """(tables, refs, moved, state); pages are moved within the pools."""
    P = len(refs)
    m = int((np.asarray(refs) > 0).sum())
    gaps, tail = [p for p in range(m) if refs[p] <= 0], [p for p in range(m, P) if refs[p] > 0]
    moved = np.array([p if refs[p] > 0 else -1 for p in range(P)], np.int32)
    out = np.array([r if p < m else 0 for p, r in enumerate(refs)], np.int32)
    for a, b in zip(tail, gaps):
        moved[a], out[b] = b, refs[a]
        for pool in pools:
            pool[b] = pool[a]
    new = np.array([[moved[p] if 0 <= p < P else p for p in row] for row in tables], np.int32).reshape(np.shape(tables))
    return new, out, moved, np.array([m, len(tail)], np.int32)


def select(logits, scores, k, history: Optional[np.ndarray] = None):
    """(scores, parents, tokens, history) in 64 bits."""
    n, beams = scores.shape
    x = np.asarray(logits, F).reshape(n, beams, -1)
    V = x.shape[2]
    total = np.full((n, beams, V), -np.inf)
    for b in range(n):
        for i in range(beams):
            row, score = x[b, i], F(scores[b, i])
            if np.isfinite(score) and not np.isnan(row).any() and np.isfinite(row.max()):
                total[b, i] = score + (row - (row.max() + np.log(np.exp(row - row.max()).sum())))
    flat = total.reshape(n, -1)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :k]
    best = np.take_along_axis(flat, order, 1)
    parents, tokens = order // V + beams * np.arange(n)[:, None], order % V
    if history is not None:
        history = np.concatenate([history[parents.reshape(-1)], tokens.reshape(-1, 1)], 1).astype(np.int32)
    return best, parents.astype(np.int32), tokens.astype(np.int32), history
