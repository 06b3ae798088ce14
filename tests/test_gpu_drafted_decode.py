"""The operators on drafts and evictions together, as a serving loop uses them: a
toy layer's tokens are decoded one by one, in drafted trees, and with a cache of
bounded size, over the block manager's tables."""
import numpy as np
import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
VOCAB, HQ, HKV, D, BS = 53, 8, 2, 64, 16


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Toy:
    """One attention layer with rotary positions: token ids in, greedy ids out."""

    def __init__(self, pk, blocks, seed):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g).to(DEV)
        self.pk, self.embed = pk, rand(VOCAB, HQ + 2 * HKV, D)
        self.out = rand(HQ * D, VOCAB) / 8
        inv, _ = pk.rope_inv_freq(D)
        self.inv = inv.to(DEV)
        self.kc, self.vc = (torch.zeros(blocks, BS, HKV, D, device=DEV) for _ in range(2))
        self.scale = D ** -0.5

    def rows(self, ids, positions):
        """Rotated q and k, and v of tokens at their positions."""
        x = self.embed[ids]
        q, k = self.pk.rope(x[:, :HQ].contiguous(), x[:, HQ:HQ + HKV].contiguous(), positions, self.inv)
        return q, k, x[:, HQ + HKV:].contiguous()

    def choose(self, o):
        n = o.shape[0]
        zero = torch.zeros(n, dtype=torch.int32, device=DEV)
        logits = (o.flatten(1) @ self.out).contiguous()
        return self.pk.sample(logits, zero.float(), zero, zero.float() + 1, zero.long(), zero.long()), logits


def tables_of(tables):
    width = max(len(t) for t in tables)
    return ints([t + [-1] * (width - len(t)) for t in tables])


def prompts(rng, n):
    return [rng.integers(0, VOCAB, int(rng.integers(3, 40))).tolist() for _ in range(n)]


def decode_one_by_one(pk, toy, seqs, steps):
    """Greedy continuation without drafts: the prompt token by token, then `steps` tokens."""
    bm = pk.BlockManager(toy.kc.shape[0], BS)
    outs = []
    for prompt in seqs:
        toks, table = [], []
        for t in range(len(prompt) + steps):
            toks.append(prompt[t] if t < len(prompt) else nxt)
            table, copy = bm.append(toks, table)
            assert copy is None
            q, k, v = toy.rows(ints([toks[-1]]).long(), torch.tensor([t], device=DEV))
            pk.kv_store_paged(k, v, tables_of([table]), ints([t + 1]), toy.kc, toy.vc)
            o = pk.paged_decode_attention(q, toy.kc, toy.vc, tables_of([table]), ints([t + 1]), t + 1, toy.scale)
            ids, logits = toy.choose(o)
            top = logits[0].topk(2).values
            assert top[0] - top[1] > 1e-4            # (30 times what fp32 sums of 512 products of an eighth differ by)
            nxt = int(ids[0])
        outs.append(toks[len(prompt):])
        bm.release(table)
    return outs


@pytest.mark.parametrize("agree", [0.0, 0.6, 1.0])
def test_drafts_change_nothing_but_the_number_of_steps(agree):
    """Trees of which some branch agrees with the target: accepted, compacted, registered -- the same tokens."""
    pk = require_gpu()
    rng = np.random.default_rng(int(agree * 10))
    toy, seqs, steps = Toy(pk, 200, 1), prompts(rng, 5), 24
    want = decode_one_by_one(pk, toy, seqs, steps)
    bm = pk.BlockManager(200, BS)
    toks, tables = [list(p[:-1]) for p in seqs], [[] for _ in seqs]
    for i, t in enumerate(toks):                     # what precedes each prompt's last token is cached
        for j in range(len(t)):
            tables[i], _ = bm.append(t[:j + 1], tables[i])
    flat = [x for t in toks for x in t]
    pos = torch.tensor([j for t in toks for j in range(len(t))], device=DEV)
    q, k, v = toy.rows(ints(flat).long(), pos)
    cu = ints(np.concatenate([[0], np.cumsum([len(t) for t in toks])]).tolist())
    pk.kv_store_prefill(k, v, tables_of(tables), cu, cu, toy.kc, toy.vc)
    roots, made, calls = [p[-1] for p in seqs], [[] for _ in seqs], 0
    while min(len(m) for m in made) < steps:
        calls += 1
        trees, drafted = [], []
        for i in range(len(seqs)):
            par, ids = [-1], [roots[i]]
            for n in range(int(rng.integers(0, 9))):
                par.append(int(rng.integers(0, len(par))))
                path, u = [], len(par) - 1
                while u > 0:
                    path.append(u)
                    u = par[u]
                k_next = len(made[i]) + len(path) - 1        # the place of this draft among the tokens to come
                right = want[i][k_next] if k_next < steps and rng.random() < agree else int(rng.integers(VOCAB))
                ids.append(right)
            trees.append(par)
            drafted.append(ids)
        old = [len(t) for t in toks]
        for i in range(len(seqs)):
            tables[i], copy = bm.reserve(old[i], len(trees[i]), tables[i])
            assert copy is None
        n = [len(t) for t in trees]
        cu_q = ints(np.concatenate([[0], np.cumsum(n)]).tolist())
        cu_k = ints(np.concatenate([[0], np.cumsum([a + b for a, b in zip(old, n)])]).tolist())
        depth = []
        for i, par in enumerate(trees):
            d = [0]
            for u in par[1:]:
                d.append(d[u] + 1)
            depth += [old[i] + x for x in d]
        ids, parents = ints([x for t in drafted for x in t]), ints([x for t in trees for x in t])
        q, k, v = toy.rows(ids.long(), torch.tensor(depth, device=DEV))
        tab, err = tables_of(tables), torch.zeros(1, dtype=torch.int32, device=DEV)
        pk.kv_store_prefill(k, v, tab, cu_q, cu_k, toy.kc, toy.vc, err=err)
        o = pk.tree_attention(q, toy.kc, toy.vc, tab, cu_q, cu_k, parents, max(n), toy.scale, err=err)
        target, _ = toy.choose(o)
        positions, first, counts, new = pk.tree_accept(ids, parents, target, cu_q, cu_k, 6, err=err)
        pk.compact_cache(toy.kc, toy.vc, tab, positions, counts, first=first, err=err)
        assert err.item() == 0 and first.tolist() == old
        for i, c in enumerate(counts.tolist()):
            got = new[i, :c].tolist()
            made[i] += got
            toks[i] += [roots[i]] + got[:-1]
            roots[i] = got[-1]
            tables[i] = bm.trim(toks[i], old[i], tables[i])
            assert len(tables[i]) == -(-len(toks[i]) // BS)
    assert [m[:steps] for m in made] == want
    assert calls < steps if agree > 0 else calls == steps or calls < steps
    if agree == 1.0:
        assert calls < 0.7 * steps
    for t in tables:
        bm.release(t)
    assert bm.num_free() == 200


def test_evictions_keep_a_cache_bounded():
    """Weights counted step by step, rows evicted and closed up: what stays gives what attention over the kept
    tokens' rows gives, head by head."""
    pk = require_gpu()
    rng = np.random.default_rng(3)
    toy, keep, limit = Toy(pk, 60, 2), 20, 33
    bm = pk.BlockManager(60, BS)
    ids = rng.integers(0, VOCAB, 90).tolist()
    other, _ = bm.allocate(ids[:7])
    table, rows, held = [], 0, [[] for _ in range(HKV)]
    weights = torch.zeros(1, HKV, limit, device=DEV)
    model = np.zeros((HKV, limit))
    xk, xv, evictions = [], [], 0
    for step, tok in enumerate(ids):
        table, copy = bm.append(ids[:rows + 1], table)
        assert copy is None
        rows += 1
        q, k, v = toy.rows(ints([tok]).long(), torch.tensor([step], device=DEV))
        xk.append(k[0].double().cpu().numpy())
        xv.append(v[0].double().cpu().numpy())
        for h in range(HKV):
            held[h].append(step)
        tab, ctx = tables_of([table]), ints([rows])
        pk.kv_store_paged(k, v, tab, ctx, toy.kc, toy.vc)
        out, _ = pk.paged_decode_attention_weights(q, toy.kc, toy.vc, tab, ctx, limit, toy.scale, weights)
        qn, got = q[0].double().cpu().numpy(), out[0].double().cpu().numpy()
        for h in range(HQ):
            kv = h // (HQ // HKV)
            K, V = np.array([xk[j][kv] for j in held[kv]]), np.array([xv[j][kv] for j in held[kv]])
            s = K @ qn[h] * toy.scale
            w = np.exp(s - s.max())
            w /= w.sum()
            # fp32 sums over at most 33 keys of unit size: 1e-5 is some 80 roundings of 2^-24
            assert np.abs(got[h] - w @ V).max() < 1e-5
            model[kv, :rows] += w
        assert np.abs(weights[0].double().cpu().numpy() - model).max() < 1e-4
        if rows == limit:
            evictions += 1
            before = weights[0].clone()
            positions, counts = pk.evict_select(weights, ctx, keep, sink=2, recent=8, weights_out=weights)
            pk.compact_cache(toy.kc, toy.vc, tab, positions, counts)
            table = bm.evict(keep, table)
            rows = int(counts[0])
            assert rows == keep and len(table) == 2
            for h in range(HKV):
                stay = positions[0, h].tolist()
                assert stay[:2] == [0, 1] and stay[-8:] == list(range(limit - 8, limit))
                assert torch.equal(weights[0, h, :keep], before[h, stay])
                held[h] = [held[h][j] for j in stay]
                model[h] = np.concatenate([model[h, stay], np.zeros(limit - keep)])
    assert evictions == 5 and held[0] != held[1]
    assert bm.allocate(ids[:40])[1] == 0             # nothing of it is taken for the prompt's blocks
    bm.release(other)
