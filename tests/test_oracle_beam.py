"""Pins of the beam oracle; the host checks of the beam entry points; the block
manager's reorder against brute force."""
import ctypes
import itertools

import numpy as np
import pytest

import oracle
from test_oracle_block_manager import ContentModel


def test_two_steps_find_the_best_pair_of_ids():
    """A beam as wide as the vocabulary loses nothing: two steps give the best pairs of a chain of brute force."""
    rng = np.random.default_rng(0)
    V = 6
    first, second = rng.normal(size=(1, V)), rng.normal(size=(V, V))
    s1, p1, t1 = oracle.beam.step(first, np.zeros(1), V)
    assert p1 == [0] * V and sorted(t1) == list(range(V)) and s1 == sorted(s1, reverse=True)
    assert abs(np.exp(s1).sum() - 1) < 1e-12
    s2, p2, t2 = oracle.beam.step(second[t1], np.array(s1), 5)
    lp1 = first[0] - np.log(np.exp(first[0]).sum())
    lp2 = second - np.log(np.exp(second).sum(1, keepdims=True))
    want = sorted(((lp1[a] + lp2[a, b], a, b) for a, b in itertools.product(range(V), range(V))), reverse=True)[:5]
    assert np.allclose(s2, [w[0] for w in want], atol=1e-12)
    assert [(t1[p], t) for p, t in zip(p2, t2)] == [(w[1], w[2]) for w in want]


def test_ties_ended_and_dead_beams():
    x = np.zeros((3, 4))
    assert oracle.beam.step(x, np.zeros(3), 5)[1:] == ([0, 0, 0, 0, 1], [0, 1, 2, 3, 0])
    s, p, t = oracle.beam.step(x, np.array([-1.0, -3.0, -np.inf]), 6, [1, 0, 0], 2)
    assert (p, t) == ([0, 1, 1, 1, 1, -1], [2, 0, 1, 2, 3, -1]) and s[0] == -1.0 and s[5] == -np.inf
    x[0, 1], x[1, 2], x[2, :3] = np.nan, np.inf, -np.inf
    s, p, t = oracle.beam.step(x, np.zeros(3), 3)
    assert (p, t) == ([2, -1, -1], [3, -1, -1]) and s[0] == 0.0
    assert oracle.beam.step(np.full((2, 3), -np.inf), np.zeros(2), 1)[1] == [-1]


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk


P = [1 << (20 + i) for i in range(8)]


def test_beam_host_checks(pk):
    L = pk.lib()
    def step(n=2, b=4, V=1000, dt=2, stride=1000, fin=None, eos=-1, keep=8, logits=P[3], scores=P[4], ws=P[5],
             wsb=1 << 30, o=P[0]):
        return L.pkvd_beam_search_step(o, P[1], P[2], logits, dt, n, b, V, stride, scores, fin, eos, keep, ws, wsb,
                                       None)
    assert step(dt=5) == 2
    assert step(n=-1) == 1
    assert step(n=0) == 0
    assert step(b=0) == 1
    assert step(b=65) == 3
    assert step(V=0) == 1
    assert step(V=(1 << 23) + 1, stride=1 << 24) == 3
    assert step(keep=0) == 1
    assert step(keep=65) == 3
    assert step(stride=999) == 1
    assert step(fin=P[6], eos=-1) == 1
    assert step(fin=P[6], eos=1000) == 1
    assert step(logits=None) == 1
    assert step(logits=P[3] + 1) == 3
    assert step(scores=None) == 1
    assert step(o=None) == 1
    assert step(ws=None) == 4
    assert step(wsb=8 * 2 * 20 - 1) == 4                    # two 1 KB chunks a row
    assert step(ws=P[5] + 4) == 3
    assert step(n=1 << 26, b=64, V=8, stride=8) == 3        # more rows than a grid holds
    size = ctypes.c_size_t(0)
    assert L.pkvd_beam_workspace_bytes(3, 4, 151936, 1, 8, ctypes.byref(size)) == 0
    assert size.value == 12 * 297 * 20                       # 297 chunks of 1 KB a row
    assert L.pkvd_beam_workspace_bytes(3, 4, 512, 1, 8, ctypes.byref(size)) == 0
    assert size.value == 12 * 20
    assert L.pkvd_beam_workspace_bytes(3, 4, 100, 0, 8, None) == 1
    assert pk.beam_workspace_bytes(0, 4, 100, __import__("torch").float32, 8) == 0


def _bytes(tables):
    return [list(t) for t in tables]


@pytest.mark.parametrize("seed", range(6))
def test_reorder_against_a_content_model(pk, seed):
    """Random beam steps: rows follow random parents, each appends its own token after the copies the manager
    asks for; every row must still read its own tokens and the counts must add up."""
    rng = np.random.default_rng(seed)
    nb, bs, B = 40, 4, 5
    bm, content = pk.BlockManager(nb, bs), ContentModel(nb, bs)
    toks = [int(t) for t in rng.integers(0, 9, 7)]
    table, _ = bm.allocate(toks)
    for p, t in enumerate(toks):
        content.write(table, p, t)
    rows = [(list(toks), list(table))] + [(list(toks), bm.fork(table)) for _ in range(B - 1)]
    for _ in range(25):
        parents = [int(x) for x in rng.integers(0, B, B)]
        if rng.random() < 0.2:
            parents = list(rng.permutation(B))
        new = bm.reorder([t for _, t in rows], parents)
        assert new == [rows[p][1] for p in parents]
        rows = [(list(rows[p][0]), t) for p, t in zip(parents, new)]
        out, copies = [], []
        for toks, table in rows:
            toks = toks + [int(rng.integers(0, 9))]
            t2, cp = bm.append(toks, table)
            assert t2 is not None
            if cp:
                copies.append(cp)
            out.append((toks, t2))
        # all copies of the step at once, before any store: no source may be another's target
        assert not {c[0] for c in copies} & {c[1] for c in copies}
        for c in copies:
            content.copy(*c)
        rows = out
        for toks, table in rows:
            content.write(table, len(toks) - 1, toks[-1])
        refs = [0] * nb
        for toks, table in rows:
            assert content.read(table, len(toks)) == toks
            for b in table:
                refs[b] += 1
        assert refs == [bm.ref_count(b) for b in range(nb)]
        assert bm.num_free() == refs.count(0)
    assert bm.reorder([t for _, t in rows], [-1] * B) == [[]] * B
    assert bm.num_free() == nb


def test_reorder_refusals_change_nothing(pk):
    bm = pk.BlockManager(8, 4)
    a, _ = bm.allocate(list(range(9)))
    b, _ = bm.allocate([50, 51])
    state = lambda: ([bm.ref_count(i) for i in range(8)], bm.num_free())
    before = state()
    for tables, parents in (([a, b], [0, 2]), ([a, b], [-2, 0]), ([a, a], [0, 1]), ([a, [7]], [0, 0]),
                            ([a, [9]], [0, 0]), ([a, [-1]], [0, 0]), ([a, [b[0], b[0]]], [0, 1])):
        with pytest.raises(pk.PkvdError):
            bm.reorder(tables, parents)
        assert state() == before
    with pytest.raises(ValueError):
        bm.reorder([a, b], [0])
    assert bm.reorder([], []) == []
    assert bm.reorder([[], a, b], [1, 0, 2]) == [a, [], b] and state() == before
    assert bm.reorder([a, b], [1, 1]) == [b, b] and bm.ref_count(b[0]) == 2 and bm.num_free() == 7
    L = pk.lib()
    i32 = lambda *v: (ctypes.c_int32 * len(v))(*v)
    t, n = i32(b[0], b[0]), i32(1, 1)
    assert L.pkvd_bm_reorder(None, i32(0, 1), 2, t, n, 1, i32(0, 0), i32(0, 0)) == 1
    assert L.pkvd_bm_reorder(bm._h, i32(0, 1), -1, t, n, 1, i32(0, 0), i32(0, 0)) == 1
    assert L.pkvd_bm_reorder(bm._h, i32(0, 1), 2, t, n, 1, t, i32(0, 0)) == 1
    assert L.pkvd_bm_reorder(bm._h, i32(0, 1), 2, t, n, 1, i32(0, 0), n) == 1
    assert L.pkvd_bm_reorder(bm._h, i32(0, 1), 2, t, i32(1, 2), 1, i32(0, 0), i32(0, 0)) == 1
    assert bm.num_free() == 7
