"""How many drafts stay: paths cut at max_path, and steps in which no draft is the target's choice."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_drafted_decode import VOCAB, Toy, decode_one_by_one, ints, prompts, tables_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cumulative(lens):
    return ints(np.concatenate([[0], np.cumsum(lens)]).tolist())


@pytest.mark.parametrize("max_path", [1, 2, 3, 31, 32, 33, 255, 256, 300])
def test_a_longer_path_is_cut(max_path):
    """Chains whose drafts are all right, some shorter than max_path, some longer, one of each length around it."""
    pk = require_gpu()
    qlen = [1, 256, 64, max(1, min(256, max_path - 1)), min(256, max_path), min(256, max_path + 1), 7]
    cached = [10 * i for i in range(len(qlen))]
    rng = np.random.default_rng(max_path)
    target = [rng.integers(0, 1000, n).tolist() for n in qlen]
    drafted = [[5] + t[:-1] for t in target]
    chains = [list(range(-1, n - 1)) for n in qlen]
    flat = lambda x: ints([v for row in x for v in row])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos, first, counts, tokens = pk.tree_accept(flat(drafted), flat(chains), flat(target), cumulative(qlen),
                                                cumulative([c + n for c, n in zip(cached, qlen)]), max_path, err=err)
    assert err.item() == 0 and first.tolist() == cached
    assert counts.tolist() == [min(n, max_path) for n in qlen]
    assert counts.max().item() == min(max_path, 256)
    for i, n in enumerate(qlen):
        m = min(n, max_path)
        assert oracle.drafts.accept(drafted[i], chains[i], target[i], max_path) == list(range(m))
        assert pos[i].tolist() == list(range(cached[i], cached[i] + m)) + [-1] * (max_path - m)
        assert tokens[i].tolist() == target[i][:m] + [-1] * (max_path - m)


def test_drafts_that_are_never_right():
    """Every step then gives its sequence one token, what decoding one by one gives, and takes all drafted blocks back."""
    pk = require_gpu()
    rng = np.random.default_rng(21)
    toy, seqs, steps = Toy(pk, 200, 1), prompts(rng, 3), 12
    want = decode_one_by_one(pk, toy, seqs, steps)
    bm = pk.BlockManager(200, 16)
    toks, tables = [list(p[:-1]) for p in seqs], [[] for _ in seqs]
    for i, t in enumerate(toks):
        for j in range(len(t)):
            tables[i], _ = bm.append(t[:j + 1], tables[i])
    pos = torch.tensor([j for t in toks for j in range(len(t))], device=DEV)
    _, k, v = toy.rows(ints([x for t in toks for x in t]).long(), pos)
    cu = cumulative([len(t) for t in toks])
    pk.kv_store_prefill(k, v, tables_of(tables), cu, cu, toy.kc, toy.vc)
    roots = [p[-1] for p in seqs]
    for step in range(steps):
        drafts = int(rng.integers(1, 20))
        old, n = [len(t) for t in toks], [1 + drafts] * len(seqs)
        for i in range(len(seqs)):
            tables[i], copy = bm.reserve(old[i], n[i], tables[i])
            assert copy is None
        # children of the root that are wrong, and below them ids that would be right there
        ids = ints([x for i in range(len(seqs)) for x in [roots[i]] + [(want[i][step] + 1 + j) % VOCAB if j < 2 else want[i][step]
                                                                    for j in range(drafts)]])
        parents = ints(([-1] + [0 if j < 2 else 1 for j in range(drafts)]) * len(seqs))
        depth = torch.tensor([old[i] + x for i in range(len(seqs)) for x in [0] + [1 if j < 2 else 2 for j in range(drafts)]],
                             device=DEV)
        cu_q, cu_k, tab = cumulative(n), cumulative([a + b for a, b in zip(old, n)]), tables_of(tables)
        q, k, v = toy.rows(ids.long(), depth)
        pk.kv_store_prefill(k, v, tab, cu_q, cu_k, toy.kc, toy.vc)
        o = pk.tree_attention(q, toy.kc, toy.vc, tab, cu_q, cu_k, parents, max(n), toy.scale)
        target, _ = toy.choose(o)
        positions, first, counts, new = pk.tree_accept(ids, parents, target, cu_q, cu_k, 4)
        pk.compact_cache(toy.kc, toy.vc, tab, positions, counts, first=first)
        assert counts.tolist() == [1] * len(seqs) and first.tolist() == old
        assert new[:, 0].tolist() == [w[step] for w in want]
        for i in range(len(seqs)):
            toks[i].append(roots[i])
            roots[i] = want[i][step]
            tables[i] = bm.trim(toks[i], old[i], tables[i])
            assert len(tables[i]) == -(-len(toks[i]) // 16)
    for t in tables:
        bm.release(t)
    assert bm.num_free() == 200
