"""The oracle of drafted trees and eviction against independent forms; the block
manager's part of both against the Python model; refusals of the C calls."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import drafts
from oracle.block_manager import BlockManager as Model


# ------------------------------------------------------------------- oracle
def test_a_node_sees_what_its_path_decoded():
    """Against PyTorch's softmax under a mask built the other way round: descendants from the top."""
    rng = np.random.default_rng(0)
    n, cached, d = 12, 9, 16
    parents = [-1, 0, 0, 1, -1, 2, 3, 3, 4, 0, 9, 8]
    K, V, q = rng.normal(size=(cached + n, d)), rng.normal(size=(cached + n, d)), rng.normal(size=(n, d))
    mask = torch.zeros(n, cached + n, dtype=torch.bool)
    mask[:, :cached] = True

    def descend(u, seen):
        mask[u, [cached + s for s in seen + [u]]] = True
        for c in range(n):
            if parents[c] == u:
                descend(c, seen + [u])
    for root in range(n):
        if parents[root] == -1:
            descend(root, [])
    s = torch.from_numpy(q @ K.T) * 0.3
    want = torch.softmax(s.masked_fill(~mask, float("-inf")), dim=1) @ torch.from_numpy(V)
    for t in range(n):
        got, _ = drafts.tree_attend(q[t], K, V, parents, t, cached, 0.3)
        assert np.allclose(got, want[t].numpy(), atol=1e-12)


def test_positions_of_nodes_are_depths():
    """A window of 2 leaves a node its parent and itself; a steep bias orders keys by depth, not by row."""
    parents = [-1, 0, 0, 2]
    V = np.eye(8)[:6]
    out, _ = drafts.tree_attend(np.zeros(4), np.zeros((6, 4)), V, parents, 3, 2, 1.0, window=2)
    assert np.allclose(out, (V[4] + V[5]) / 2)
    out, _ = drafts.tree_attend(np.zeros(4), np.zeros((6, 4)), V, parents, 3, 2, 1.0, slope=np.log(2.0))
    w = np.array([2.0 ** -4, 2.0 ** -3, 2.0 ** -2, 0, 2.0 ** -1, 1.0])
    assert np.allclose(out[:6], w / w.sum())


def test_accept_by_hand():
    parents = [-1, 0, 0, 1, 2, 2, 4]
    drafted = [9, 5, 5, 7, 6, 8, 1]
    assert drafts.accept(drafted, parents, [5, 7, 8, 0, 0, 0, 0], 9) == [0, 1, 3]     # the lowest of two children
    assert drafts.accept(drafted, parents, [5, 1, 8, 0, 0, 0, 0], 9) == [0, 1]
    assert drafts.accept(drafted, parents, [4, 0, 0, 0, 0, 0, 0], 9) == [0]
    assert drafts.accept(drafted, parents, [5, 7, 0, 0, 0, 0, 0], 2) == [0, 1]
    assert drafts.accept([], [], [], 3) == []


def test_stays_by_brute_force():
    rng = np.random.default_rng(1)
    for _ in range(200):
        n, keep = int(rng.integers(0, 30)), int(rng.integers(1, 12))
        sink = int(rng.integers(0, keep + 1))
        recent = int(rng.integers(0, keep - sink + 1))
        w = rng.integers(0, 4, 30) / 2
        got = drafts.stays(w, n, keep, sink, recent)
        assert got == sorted(set(got)) and len(got) == min(n, keep)
        if n <= keep:
            continue
        inside = [j for j in range(n) if j < sink or j >= n - recent]
        assert set(inside) <= set(got)
        out = [j for j in range(n) if j not in got]
        chosen = [j for j in got if j not in inside]
        assert all(w[a] > w[b] or (w[a] == w[b] and a < b) for a in chosen for b in out)


def test_given_sums_to_one_and_matches_attend():
    rng = np.random.default_rng(2)
    K, q = rng.normal(size=(40, 8)), rng.normal(size=8)
    w, bound = drafts.given(q, K, 40, 0.5, cap=3.0, slope=0.1, window=13)
    assert abs(w.sum() - 1) < 1e-12 and np.all(w[:27] == 0) and np.all(bound > 0) and np.all(bound[27:] < 1e-4)
    out, _ = oracle.scores.attend(q, K, np.eye(40), 39, 0.5, 3.0, 0.1, 13)
    assert np.allclose(out, w)


# ------------------------------------------------------------ block manager
@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk


def same(bm, model, blocks):
    assert bm.num_free() == model.num_free()
    assert [bm.ref_count(b) for b in range(blocks)] == model.ref


def test_block_manager_against_the_model(pk):
    """Random prompts, appends, forks, drafts and evictions: the same tables, references and free blocks."""
    nb, bs = 40, 4
    rng = np.random.default_rng(3)
    bm, model = pk.BlockManager(nb, bs), Model(nb, bs)
    live = []                                    # [tokens, table]
    seen = {k: 0 for k in ("allocate", "append", "fork", "draft", "evict", "release", "full", "copy")}
    for _ in range(3000):
        op = str(rng.choice(["allocate", "append", "fork", "draft", "draft", "evict", "release"]))
        if op == "allocate":
            toks = rng.integers(0, 2, int(rng.integers(1, 20))).tolist()
            got, want = bm.allocate(toks), model.allocate(toks)
            assert got == want
            if got:
                live.append([toks, got[0]])
        elif live:
            i = int(rng.integers(len(live)))
            toks, table = live[i]
            if op == "append":
                new = toks + [int(rng.integers(2))]
                got, want = bm.append(new, table), model.append(new, table)
                assert got == want
                if got[0] is not None:
                    live[i] = [new, got[0]]
            elif op == "fork":
                bm.fork(table), model.fork(table)
                live.append([list(toks), list(table)])
            elif op == "draft":
                n = int(rng.integers(0, 11))
                got, want = bm.reserve(len(toks), n, table), model.reserve(len(toks), n, table)
                assert got == want
                if got[0] is None:
                    seen["full"] += 1
                else:
                    same(bm, model, nb)
                    seen["copy"] += got[1] is not None
                    new = toks + rng.integers(0, 2, int(rng.integers(0, n + 1))).tolist()
                    a, b = bm.trim(new, len(toks), got[0]), model.trim(new, len(toks), got[0])
                    assert a == b
                    live[i] = [new, a]
            elif op == "evict":
                keep = int(rng.integers(1, len(toks) + 1))
                if any(model.ref[b] != 1 for b in table):
                    with pytest.raises(pk.PkvdError):
                        bm.evict(keep, table)
                    continue
                a, b = bm.evict(keep, table), model.evict(keep, table)
                assert a == b
                live[i] = [toks[:keep], a]
            else:
                bm.release(table), model.release(table)
                live.pop(i)
        seen[op] += 1
        same(bm, model, nb)
    assert min(seen.values()) > 20, seen


def test_evicted_rows_are_no_prompts(pk):
    """Neither what an eviction leaves nor what is appended behind it is found by a later prompt."""
    bm = pk.BlockManager(30, 4)
    prompt = list(range(13))
    table, _ = bm.allocate(prompt)
    table = bm.evict(6, table)
    assert len(table) == 2
    toks = prompt[:6]
    for t in range(6, 12):
        toks.append(t)
        table, copy = bm.append(toks, table)
        assert copy is None
    assert bm.allocate(prompt)[1] == 0           # the same ids as the appended ones, and none is cached
    bm.release(table)
    again, cached = bm.allocate(prompt)
    assert cached == 12                          # the second prompt's blocks are


def test_accepted_drafts_are_found_by_later_prompts(pk):
    bm = pk.BlockManager(30, 4)
    table, _ = bm.allocate([1, 2, 3])
    table, copy = bm.reserve(3, 9, table)
    assert len(table) == 3 and copy is None and bm.num_free() == 27
    table = bm.trim([1, 2, 3, 4, 5, 6, 7, 8], 3, table)
    assert len(table) == 2 and bm.num_free() == 28
    assert bm.allocate([1, 2, 3, 4, 5, 6, 7, 8, 9])[1] == 8


def test_a_shared_sequence_is_cut_into_fresh_blocks(pk):
    bm = pk.BlockManager(10, 4)
    table, _ = bm.allocate(list(range(8)))
    other = bm.fork(table)
    with pytest.raises(pk.PkvdError):
        bm.evict(5, table)
    assert bm.num_free() == 8
    fresh, copy = bm.reserve(0, 5, [])
    assert copy is None and len(fresh) == 2 and not set(fresh) & set(table)
    assert bm.evict(5, fresh) == fresh
    bm.release(table)
    assert [bm.ref_count(b) for b in other] == [1, 1]


def test_block_manager_refusals(pk):
    bm = pk.BlockManager(4, 4)
    table, _ = bm.allocate([1, 2, 3, 4, 5])
    free = bm.num_free()
    assert bm.reserve(5, 100, table) == (None, None)
    for bad in (lambda: bm.reserve(9, 1, table), lambda: bm.reserve(-1, 1, table), lambda: bm.reserve(5, -1, table),
                lambda: bm.reserve(5, 1, [table[0], 99]), lambda: bm.trim([1] * 9, 5, table), lambda: bm.trim([1, 2], 5, table),
                lambda: bm.evict(0, table), lambda: bm.evict(9, table), lambda: bm.evict(2, [3, 77])):
        with pytest.raises(pk.PkvdError):
            bad()
    assert bm.num_free() == free and [bm.ref_count(b) for b in table] == [1, 1]


# ----------------------------------------------------------------- refusals
OK, INVALID, DTYPE, SHAPE, SMALL = 0, 1, 2, 3, 4
P = 1 << 20              # an aligned address that is never read


def cache(capi, **kw):
    c = capi.PkvdCache(P, P, 2, 16, 64, 8, 128, 16 * 8 * 128, 8 * 128, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def call(fn, order, defaults, **kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    a = dict(defaults, **kw)
    return fn(*[a[k] for k in order.split()])


TREE = "out q cache tables max_blocks cu_q cu_k parents seqs total max_q hq scale window mod ws ws_bytes stream err path"


def test_tree_attention_refusals(pk):
    from paged_kv_decode_store_gb300 import _capi
    L = pk.lib()
    base = dict(out=P, q=P, cache=cache(_capi), tables=P, max_blocks=8, cu_q=P, cu_k=P, parents=P, seqs=0, total=20, max_q=9,
                hq=48, scale=0.1, window=0, mod=None, ws=None, ws_bytes=0, stream=None, err=None, path=0)
    go = lambda **kw: call(L.pkvd_tree_attention, TREE, base, **kw)
    assert go() == OK and go(seqs=3, total=0) == OK and go(seqs=3, max_q=0) == OK
    for kw in (dict(seqs=-1), dict(total=-1), dict(max_q=-1), dict(window=-1), dict(scale=float("nan")), dict(path=9), dict(hq=0),
               dict(mod=_capi.PkvdScoreMod(-1.0, None, None)), dict(mod=_capi.PkvdScoreMod(0.0, None, P)),
               dict(cache=cache(_capi, k_base=0)), dict(seqs=2, q=None), dict(seqs=2, parents=None), dict(seqs=2, max_blocks=0), dict(seqs=2)):
        assert go(**kw) == INVALID, kw
    for kw in (dict(hq=44), dict(hq=8 * 129), dict(max_q=257), dict(seqs=65536), dict(path=2), dict(cache=cache(_capi, head_dim=96)),
               dict(cache=cache(_capi, block_size=24)), dict(seqs=2, q=P + 8), dict(seqs=2, out=P + 4)):
        assert go(**kw) == SHAPE, kw
    assert go(cache=cache(_capi, dtype=7)) == DTYPE and go(cache=cache(_capi, dtype=0), path=3) == DTYPE
    n = ctypes.c_size_t(0)
    size = lambda *a: (L.pkvd_tree_workspace_bytes(*a, ctypes.byref(n)), n.value)
    assert size(4, 48, 8, 128, 9, 152)[0] == OK and 0 < size(4, 48, 8, 128, 9, 152)[1] < size(4, 48, 8, 128, 200, 152)[1] < 64 << 20
    assert size(4, 48, 8, 128, 0, 152) == (OK, 0)
    assert size(4, 47, 8, 128, 9, 152)[0] == SHAPE and size(4, 48, 8, 128, 257, 152)[0] == SHAPE
    assert size(-1, 48, 8, 128, 9, 152)[0] == INVALID and size(4, 48, 0, 128, 9, 152)[0] == INVALID


def test_tree_accept_refusals(pk):
    L = pk.lib()
    order = "positions first counts tokens drafted parents target cu_q cu_k seqs total max_path stream err"
    base = {k: P for k in order.split()}
    base.update(seqs=0, total=10, max_path=4, stream=None, err=None)
    go = lambda **kw: call(L.pkvd_tree_accept, order, base, **kw)
    assert go() == OK
    for kw in (dict(seqs=-1), dict(total=-1), dict(max_path=0), dict(seqs=2, positions=None), dict(seqs=2, first=None),
               dict(seqs=2, counts=None), dict(seqs=2, tokens=None), dict(seqs=2, cu_q=None), dict(seqs=2, drafted=None)):
        assert go(**kw) == INVALID, kw


def test_compact_refusals(pk):
    from paged_kv_decode_store_gb300 import _capi
    L = pk.lib()
    order = "cache tables max_blocks new new_blocks positions stride head_stride counts first seqs most stream err"
    base = {k: P for k in order.split()}
    base.update(cache=cache(_capi), max_blocks=8, new_blocks=8, stride=100, head_stride=0, seqs=0, most=100, stream=None, err=None,
                first=None)
    go = lambda **kw: call(L.pkvd_compact_cache, order, base, **kw)
    assert go() == OK and go(seqs=2, most=0) == OK
    for kw in (dict(seqs=-1), dict(most=-1), dict(stride=-1), dict(head_stride=-1), dict(seqs=2, tables=None), dict(seqs=2, new=None),
               dict(seqs=2, positions=None), dict(seqs=2, counts=None), dict(seqs=2, max_blocks=0), dict(seqs=2, new_blocks=0),
               dict(seqs=2, new_blocks=9), dict(cache=cache(_capi, v_base=0))):
        assert go(**kw) == INVALID, kw
    assert go(seqs=65536) == SHAPE and go(cache=cache(_capi, block_size=12)) == SHAPE and go(cache=cache(_capi, dtype=5)) == DTYPE


WEIGHTS = ("out q cache tables max_blocks ctx most seqs hq scale window mod w_out w s_seq s_head heads ws ws_bytes stream err "
           "path")


def test_weights_refusals(pk):
    from paged_kv_decode_store_gb300 import _capi
    L = pk.lib()
    base = {k: P for k in WEIGHTS.split()}
    base.update(cache=cache(_capi), max_blocks=8, most=100, seqs=0, hq=48, scale=0.1, window=0, mod=None, s_seq=800, s_head=100,
                heads=8, ws=None, ws_bytes=0, stream=None, err=None, path=0)
    go = lambda **kw: call(L.pkvd_paged_decode_attention_weights, WEIGHTS, base, **kw)
    assert go() == OK and go(heads=1) == OK
    for kw in (dict(heads=2), dict(heads=48), dict(window=-1), dict(seqs=-1), dict(scale=float("inf")),
               dict(window=5, mod=_capi.PkvdScoreMod(0.0, None, P)), dict(mod=_capi.PkvdScoreMod(float("nan"), None, None))):
        assert go(**kw) == INVALID, kw
    assert go(hq=72) == SHAPE and go(path=3) == SHAPE and go(cache=cache(_capi, block_size=8)) == SHAPE
    n, m = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert L.pkvd_decode_weights_workspace_bytes(4, 48, 128, 1001, 152, ctypes.byref(n)) == OK
    assert L.pkvd_decode_workspace_bytes(4, 48, 128, 1001, 152, ctypes.byref(m)) == OK
    assert n.value >= m.value + 4 * 48 * (4 * 1001 + 8)
    assert L.pkvd_decode_weights_workspace_bytes(4, 48, 128, -1, 152, ctypes.byref(n)) == INVALID


def test_select_refusals(pk):
    L = pk.lib()
    order = "positions counts w_out w s_seq s_head length ctx seqs heads keep sink recent stream err"
    base = {k: P for k in order.split()}
    base.update(s_seq=800, s_head=100, length=100, seqs=0, heads=8, keep=10, sink=2, recent=8, stream=None, err=None)
    go = lambda **kw: call(L.pkvd_evict_select, order, base, **kw)
    assert go() == OK
    for kw in (dict(seqs=-1), dict(heads=0), dict(length=0), dict(keep=0), dict(sink=-1), dict(recent=-1), dict(sink=3),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(seqs=2, s_seq=99), dict(seqs=2, s_head=99), dict(seqs=2, w=None),
               dict(seqs=2, positions=None), dict(seqs=2, counts=None), dict(seqs=2, ctx=None)):
        assert go(**kw) == INVALID, kw
    assert go(seqs=65536) == SHAPE and go(seqs=2, w=P + 2) == SHAPE
