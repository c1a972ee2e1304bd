"""TEST INFRASTRUCTURE ONLY: verification of drafted tokens, row by row in fp64 numpy."""
from __future__ import annotations

import numpy as np


def _clean(x):
    x = np.asarray(x, np.float64)
    return np.where((x > 0) & (x < np.inf), x, 0.0)


def verify(target, tokens, u, u_draw, draft=None, n_draft=None):
    """(out [B, N+1], kept [B]) of arrays: target [B, N+1, vocab], draft [B, N, vocab] or None."""
    with np.errstate(invalid="ignore"):
        target = _clean(target)
        draft = None if draft is None else _clean(draft)
    u, u_draw, tokens = np.asarray(u, np.float64), np.asarray(u_draw, np.float64), np.asarray(tokens)
    B, places, vocab = target.shape
    N = places - 1
    out, kept = np.full((B, places), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        given = N if n_draft is None else min(max(int(n_draft[b]), 0), N)
        n = 0
        while n < given:
            x = int(tokens[b, n])
            if not 0 <= x < vocab:
                break
            q = 1.0 if draft is None else draft[b, n, x]
            if not u[b, n] * q < target[b, n, x]:
                break
            out[b, n] = x
            n += 1
        weight = target[b, n].copy()
        if n < given:
            if draft is not None:
                weight -= draft[b, n]
            elif 0 <= tokens[b, n] < vocab:
                weight[tokens[b, n]] -= 1.0
            weight = np.maximum(weight, 0.0)
            if not weight.any():
                weight = target[b, n]
        if weight.any():
            upto = np.cumsum(weight)
            past = np.flatnonzero((upto > u_draw[b] * upto[-1]) & (weight > 0))
            out[b, n] = past[0] if past.size else np.flatnonzero(weight)[-1]
        kept[b] = n + 1
    return out, kept
