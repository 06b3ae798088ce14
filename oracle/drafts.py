"""Trees of drafted tokens and eviction in float64 (test oracle).

TEST INFRASTRUCTURE ONLY.

Tree attention: node t of a tree behind `cached` tokens sees what a decode step
would see that had decoded its path: the cached tokens, its ancestors in order,
itself.  So its result is that of ``scores.attend`` over exactly those keys, at
position cached + depth.

Accept: the path of nodes whose drafted ids are the target's choices.

Eviction: of a sequence longer than `keep` stay the first `sink`, the last
`recent` and the heaviest of the others, the lowest position first among equals.

Weights: what a decode step gives each key, with a bound counted from the
roundings as in ``scores.attend``.
"""
from __future__ import annotations

import numpy as np

from . import scores


def path_of(parents, t: int) -> list[int]:
    """Nodes from the root's side down to t."""
    path = []
    while t >= 0:
        path.append(t)
        t = int(parents[t])
    return path[::-1]


def tree_attend(q, K, V, parents, t: int, cached: int, scale: float, **kw):
    """(output [D], bound [D]) of node t over K, V [cached + nodes, D] (kw: as scores.attend)."""
    keys = list(range(cached)) + [cached + u for u in path_of(parents, t)]
    return scores.attend(q, K[keys], V[keys], len(keys) - 1, scale, **kw)


def accept(drafted, parents, target, max_path: int) -> list[int]:
    """The accepted nodes of one tree."""
    if len(drafted) == 0:
        return []
    path = [0]
    while len(path) < max_path:
        here = path[-1]
        nxt = [c for c in range(here + 1, len(drafted)) if parents[c] == here and drafted[c] == target[here]]
        if not nxt:
            break
        path.append(nxt[0])
    return path


def stays(weights, n: int, keep: int, sink: int, recent: int) -> list[int]:
    """Positions of a sequence of n tokens that stay."""
    if n <= keep:
        return list(range(n))
    middle = range(sink, n - recent)
    def heavier_first(j):
        w = float(weights[j])
        return (0, 0.0, j) if np.isnan(w) else (1, -w, j)
    chosen = sorted(middle, key=heavier_first)[:keep - sink - recent]
    return sorted(list(range(sink)) + chosen + list(range(n - recent, n)))


def given(q, K, n: int, scale: float, cap: float = 0.0, slope: float = 0.0, window: int = 0,
          cap_error: float = scores.CAP_ERROR["16-bit"]):
    """(softmax weights [n], bound [n]) of a decode step's query over its n keys."""
    seen = scores.visible_keys(n - 1, n, window)
    j = np.arange(n)
    s = scale * (K[:n].astype(np.float64) @ q)
    err = abs(scale) * (np.abs(K[:n]) @ np.abs(q)) * 2.0 ** -24 * (q.shape[0] + 2)
    if cap > 0:
        s = cap * np.tanh(s / cap)
        err = err + np.abs(s) * cap_error
    s = s - slope * (n - 1 - j)
    s = np.where(seen, s, -np.inf)
    top = s.max()
    w = np.exp(s - top)
    w = w / w.sum()
    near = np.where(seen, np.abs(s), 0.0)
    e = err + (near + abs(top) + abs(slope) * (n - 1 - j)) * 4 * 2.0 ** -24 + 2.0 ** -22
    e = np.where(seen, e, 0.0)
    total = (w * e).sum() + n * 2.0 ** -24           # of the sum, relative
    return w, 2 * w * (e + total) + 2.0 ** -126      # a weight below fp32's normal range may be flushed
