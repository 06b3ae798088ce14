"""Seeded random shapes of drafted trees, of decode with weights, of the
selection and the moves of cached rows against the float64 oracles: head counts
and groups, types, block sizes, batches of one to hundreds, lengths from nothing
to thousands, caps, slopes and windows."""
import numpy as np
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_eviction import DEV, a_cache, bits, ints, moved, run_select, run_weights
from test_gpu_score_mod import DT
from test_gpu_tree import run_tree

pytestmark = pytest.mark.gpu


def modifiers(rng, windows):
    kind = [None, None, "geometric", "mixed"][int(rng.integers(0, 4))]
    return float(rng.choice([0, 0, 0, 5, 30])), kind, int(rng.choice(windows))


def random_tree(pk, seed):
    rng = np.random.default_rng(seed)
    hkv, group = int(rng.choice([1, 2, 3, 4, 8])), int(rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 33, 48, 64, 100, 128]))
    if hkv * group > 256:
        hkv = 1
    dt, d = str(rng.choice(["bf16", "f16", "f32", "bf16", "f16"])), int(rng.choice([64, 128]))
    bs = int(rng.choice([8, 16, 32, 64, 128, 256]))
    path = int(rng.choice([0, 1] if dt == "f32" else [0, 0, 0, 1, 3]))
    seqs, most = int(rng.choice([1, 2, 3, 5, 9, 40, 140])), int(rng.choice([1, 2, 5, 9, 17, 33, 64, 65, 130, 256]))
    if group > 16:
        seqs, most = min(seqs, 9), min(most, 33)
    if seqs > 9:
        most = min(most, 9)
    qlen = [int(rng.integers(0, most + 1)) for _ in range(seqs)]
    qlen[int(rng.integers(0, seqs))] = most
    longest = int(rng.choice([1, 50, 130, 400, 1500])) if seqs <= 9 else 200
    cached = [int(rng.integers(0, longest + 1)) for _ in range(seqs)]
    run_tree(pk, (dt, hkv * group, hkv, d, bs, path), qlen, cached, modifiers(rng, [0, 0, 0, 1, 3, 40, 128, 200, 1000]),
             seed=seed, every=max(1, sum(qlen) * hkv * group // 150))


def random_select(pk, seed):
    rng = np.random.default_rng(seed)
    seqs, heads = int(rng.choice([1, 2, 7, 45, 300])), int(rng.choice([1, 2, 8]))
    length = int(rng.choice([1, 3, 31, 64, 500, 4097, 30000])) if seqs < 3 else int(rng.choice([1, 31, 64, 150, 700]))
    w = torch.empty(seqs, heads, length).exponential_(1.0, generator=torch.Generator().manual_seed(seed)) ** int(rng.choice([1, 4]))
    if rng.random() < 0.3:
        w = torch.round(w * 4) / 4
    keep = int(rng.integers(1, length + 5))
    sink = int(rng.integers(0, min(keep, 9) + 1))
    recent = int(rng.integers(0, keep - sink + 1))
    run_select(pk, w, [int(rng.integers(0, length + 1)) for _ in range(seqs)], keep, sink, recent, bool(rng.integers(0, 2)))


def random_weights(pk, seed):
    rng = np.random.default_rng(seed)
    dt = str(rng.choice(["bf16", "f16", "f32"]))
    hkv, group = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 2, 3, 5, 6, 8]))
    d, bs = 64 if dt == "f32" else int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 256]))
    ctx = [int(x) for x in rng.choice([0, 1, 2, 15, 16, 17, 63, 130, 257, 600], size=int(rng.integers(1, 9)))]
    run_weights(pk, (dt, hkv * group, hkv, d, bs, 0), ctx, modifiers(rng, [0, 0, 1, 40, 200]),
                heads=int(rng.choice([1, hkv])), seed=seed, every=max(1, hkv * group // 6), slack=int(rng.integers(0, 9)))


def random_compact(pk, seed):
    rng = np.random.default_rng(seed)
    dt, hkv, d = str(rng.choice(["bf16", "f16", "f32"])), int(rng.choice([1, 2, 3, 8])), int(rng.choice([64, 128]))
    bs, seqs, fresh = int(rng.choice([1, 8, 16, 64, 256])), int(rng.integers(1, 9)), bool(rng.integers(0, 2))
    longest = int(rng.choice([3, 20, 40, 300, 900]))
    lens = rng.integers(1, longest + 1, seqs)
    first = np.array([int(rng.integers(0, n)) for n in lens]) * int(rng.integers(0, 2))
    counts = np.array([int(rng.integers(0, n - f + 1)) for n, f in zip(lens, first)])
    heads = int(rng.choice([0, 1, hkv]))                       # 0: positions [S, n]
    pos = np.full((seqs, max(heads, 1), max(int(counts.max()), 1)), -1)
    for i in range(seqs):
        for h in range(max(heads, 1)):
            pos[i, h, :counts[i]] = np.sort(rng.choice(np.arange(first[i], lens[i]), counts[i], replace=False))
    need = -(-lens // bs)
    blocks = 2 * int(need.sum()) + 2
    cut = np.split(rng.permutation(blocks)[:2 * int(need.sum())], np.cumsum(np.concatenate([need, need]))[:-1])
    tables = [np.full((seqs, int(need.max())), -1) for _ in range(2)]
    for i in range(seqs):
        for t in range(2):
            tables[t][i, :need[i]] = cut[t * seqs + i]
    if not fresh:
        tables[1] = tables[0]
    kc, vc = a_cache(blocks, bs, hkv, d, DT[dt], seed)
    if heads == 0:
        pos = pos[:, 0]
    want = [moved(c, tables[0], tables[1], pos, counts, first, bs) for c in (kc, vc)]
    dev = [torch.tensor(t, dtype=torch.int32, device=DEV) for t in tables]
    err = ints([0])
    pk.compact_cache(kc, vc, dev[0], torch.tensor(pos, dtype=torch.int32, device=DEV), ints(counts.tolist()),
                     first=ints(first.tolist()), new_tables=dev[1] if fresh else None, err=err)
    assert err.item() == 0
    for c, w in zip((kc, vc), want):
        assert np.array_equal(bits(c), w)


@pytest.mark.parametrize("seed", range(24))
def test_trees(seed):
    random_tree(require_gpu(), seed)


@pytest.mark.parametrize("seed", range(16))
def test_selection(seed):
    random_select(require_gpu(), seed)


@pytest.mark.parametrize("seed", range(16))
def test_weights(seed):
    random_weights(require_gpu(), seed)


@pytest.mark.parametrize("seed", range(16))
def test_moves(seed):
    random_compact(require_gpu(), seed)
