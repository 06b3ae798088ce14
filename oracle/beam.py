"""One step of beam search in float64 (test oracle).

TEST INFRASTRUCTURE ONLY.  The value of continuing beam b of a request with id
j is scores[b] + x_bj - log(sum_i exp x_bi).  The `keep` largest are kept, best
first, the lowest b * V + j first among equal ones.  An ended beam continues
with its end id alone, at its score.  A beam whose score or normaliser is not
finite offers nothing, an id at -inf is never chosen; where there are fewer
than `keep` continuations: (-inf, -1, -1).
"""
from __future__ import annotations

import numpy as np


def log_softmax(x: np.ndarray):
    """x - log sum exp x (from the largest x: rows of huge numbers keep their
    sum), or None if the normaliser is not finite."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
        return None
    m = x.max()
    return (x - m) - np.log(np.exp(x - m).sum())


def step(logits: np.ndarray, scores: np.ndarray, keep: int, finished=None, eos_id: int = -1):
    """logits [B, V], scores [B] of one request -> (scores, parents, tokens) lists of length keep."""
    B, V = logits.shape
    value = np.full((B, V), -np.inf)
    for b in range(B):
        s = float(scores[b])
        if not np.isfinite(s):
            continue
        if finished is not None and finished[b]:
            value[b, eos_id] = s
            continue
        lp = log_softmax(logits[b])
        if lp is not None:
            value[b] = s + lp
    flat = value.ravel()
    order = np.argsort(-flat, kind="stable")[:keep]
    out = [(flat[i], int(i) // V, int(i) % V) if flat[i] > -np.inf else (-np.inf, -1, -1) for i in order]
    out += [(-np.inf, -1, -1)] * (keep - len(out))
    return [o[0] for o in out], [o[1] for o in out], [o[2] for o in out]
