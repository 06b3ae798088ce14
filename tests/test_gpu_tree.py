"""Attention of drafted trees over the paged cache, both paths, against the
float64 oracle within its counted bound; and which drafts stay, exactly."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_score_mod import DT, cache_of, slopes_for, tolerances

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def cumulative(lens):
    return ints(np.concatenate([[0], np.cumsum(lens)]).tolist())


def a_tree(n, kind, rng):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "forest":                     # several nodes follow the cache directly
        return [-1 if rng.random() < 0.3 else int(rng.integers(-1, t)) for t in range(n)]
    return [-1] + [int(rng.integers(max(0, t - 4), t)) for t in range(1, n)] if n else []


KINDS = ["tree", "chain", "star", "forest"]


def run_tree(pk, case, qlen, cached, mod=(0.0, None, 0), seed=0, every=1, max_q=None, workspace=None):
    """One call against the oracle; every `every`-th (row, head) is looked at."""
    dt, hq, hkv, d, bs, path = case
    dt = DT[dt]
    cap, kind, window = mod
    rng = np.random.default_rng(seed)
    klen = [c + n for c, n in zip(cached, qlen)]
    kc, vc, tables, rows = cache_of(klen, hkv, d, bs, dt, seed)
    trees = [a_tree(n, KINDS[i % 4], rng) for i, n in enumerate(qlen)]
    T, tail = sum(qlen), 3
    q = (3 * torch.randn(T + tail, hq, d, generator=torch.Generator().manual_seed(seed + 1))).to(dt)
    dev_slopes, slopes = slopes_for(hq, kind)
    scale, err = d ** -0.5, torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((T + tail, hq, d), 7.0, dtype=dt, device=DEV)
    pk.tree_attention(q.to(DEV), kc, vc, tables, cumulative(qlen), cumulative(klen),
                      ints([u for t in trees for u in t] + [-1] * tail), max_q or max(qlen), scale, window=window,
                      out=out, err=err, path=path, softcap=cap, alibi_slopes=dev_slopes, workspace=workspace)
    assert err.item() == 0
    assert torch.all(out[T:] == 7.0)         # rows behind the last sequence
    got = out.double().cpu().numpy()
    tensor = dt != torch.float32 and path != pk.PATH_FMA
    tol = tolerances(dt, tensor)
    t = count = 0
    for i, n in enumerate(qlen):
        for j in range(n):
            for h in range(hq):
                count += 1
                if count % every:
                    continue
                k, v = (x[:, h // (hq // hkv)] for x in rows[i])
                want, bound = oracle.drafts.tree_attend(q[t, h].double().numpy(), k, v, trees[i], j, cached[i], scale,
                                                        cap=cap, slope=slopes[h], window=window, **tol)
                off = np.abs(got[t, h] - want)
                assert np.all(off <= bound), (i, j, h, float((off - bound).max()))
            t += 1
    return out


LAYOUTS = [  # dtype, hq, hkv, d, bs, path
    ("f32", 4, 2, 64, 16, 0), ("f32", 6, 1, 128, 32, 0), ("bf16", 48, 8, 128, 16, 0), ("f16", 16, 16, 64, 256, 0),
    ("f16", 5, 1, 128, 64, 3), ("bf16", 64, 8, 64, 16, 3), ("bf16", 12, 4, 128, 128, 1), ("f16", 8, 8, 64, 8, 1),
    ("f16", 6, 2, 64, 8, 3),
]
MODS = [(0.0, None, 0), (5.0, None, 0), (0.0, "geometric", 0), (2.0, "mixed", 0), (0.0, None, 37), (30.0, "mixed", 150),
        (0.0, "mixed", 3)]


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("case", LAYOUTS, ids=lambda c: "-".join(map(str, c)))
def test_layouts(case, mod):
    """Trees of one node to more than a Q tile, contexts of nothing, of whole tiles and of odd lengths."""
    pk = require_gpu()
    run_tree(pk, case, [1, 0, 7, 33, 1, 16], [0, 40, 126, 301, 128, 0], mod, every=7 if case[1] > 8 else 2)


@pytest.mark.parametrize("case", [("bf16", 64, 8, 128, 16, 3), ("f16", 2, 2, 64, 16, 3), ("bf16", 128, 1, 64, 16, 3),
                                  ("f32", 2, 1, 64, 16, 1), ("f16", 96, 2, 128, 32, 3)],
                         ids=lambda c: "-".join(map(str, c)))
def test_units(case):
    """Trees of several units: many nodes, many query heads a KV head; the drafted keys cross tiles."""
    pk = require_gpu()
    most = 200 if case[1] // case[2] < 16 else 40
    run_tree(pk, case, [most, 3, 65, 129 if most == 200 else 9], [100, 1000, 383, 2], (0.0, "mixed", 0), seed=3, every=37)


def test_largest_tree():
    pk = require_gpu()
    run_tree(pk, ("bf16", 4, 1, 64, 16, 3), [256, 256], [0, 513], (3.0, None, 90), seed=4, every=11)


def test_long_context_in_many_pieces():
    """Few rows over a long context: every CTA has a piece, the merge joins them by eight warps a row."""
    pk = require_gpu()
    run_tree(pk, ("bf16", 3, 1, 128, 16, 3), [4], [40000], seed=5)
    run_tree(pk, ("f16", 2, 2, 64, 64, 3), [2, 1], [30011, 9], (20.0, None, 0), seed=6)
    run_tree(pk, ("f32", 2, 1, 64, 64, 1), [3], [9000], seed=7)


@pytest.mark.parametrize("path", [1, 3])
def test_many_short_sequences(path):
    """More sequences than threads, one tile of keys each: one stream idles, slices hold many segments."""
    pk = require_gpu()
    rng = np.random.default_rng(8)
    qlen = rng.integers(0, 4, 700).tolist()
    cached = rng.integers(0, 150, 700).tolist()
    run_tree(pk, ("bf16", 4, 2, 64, 16, path), qlen, cached, (0.0, "geometric", 0), seed=8, every=5)


@pytest.mark.parametrize("path", [1, 3])
@pytest.mark.parametrize("seqs", [32, 33, 128, 129])
def test_batches_around_a_warp_and_its_plan(seqs, path):
    """Slices that every CTA finds by itself and those of a plan, with empty sequences at both ends and between."""
    pk = require_gpu()
    rng = np.random.default_rng(seqs)
    qlen = rng.integers(0, 6, seqs)
    qlen[[0, seqs // 2, seqs - 1]] = 0
    qlen[1], qlen[seqs - 2] = 5, 3
    cached = rng.integers(0, 600, seqs)
    run_tree(pk, ("f16", 4, 2, 64, 16, path), qlen.tolist(), cached.tolist(), (0.0, None, 0), seed=seqs, every=3)


def test_max_seqlen_above_every_tree():
    pk = require_gpu()
    run_tree(pk, ("bf16", 16, 2, 128, 16, 3), [3, 1], [50, 300], seed=9, max_q=256)


def setup(pk, dt=torch.bfloat16, hq=16, hkv=2, d=128, bs=16, qlen=(9, 4), cached=(200, 700), seed=11):
    klen = [c + n for c, n in zip(cached, qlen)]
    kc, vc, tables, _ = cache_of(klen, hkv, d, bs, dt, seed)
    rng = np.random.default_rng(seed)
    parents = ints([u for n in qlen for u in a_tree(n, "tree", rng)])
    q = torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(seed)).to(dt).to(DEV)
    return dict(q=q, k_cache=kc, v_cache=vc, block_tables=tables, cu_seqlens_q=cumulative(qlen),
                cu_seqlens_k=cumulative(klen), parents=parents, max_seqlen_q=max(qlen), scale=d ** -0.5)


@pytest.mark.parametrize("path", [1, 3])
def test_a_chain_is_causal_attention(path):
    """Chained drafts are the rows of a causal prefill chunk: the two calls agree within their roundings."""
    pk = require_gpu()
    a = setup(pk)
    a["parents"] = ints(list(range(-1, 8)) + list(range(-1, 3)))
    tree = pk.tree_attention(**a, path=path)
    del a["parents"]
    plain = pk.prefill_attention(**a, path=path)
    # two calls, each: half a step a weight in sum and normaliser, half a step of the output
    a["v_cache"] = a["v_cache"].abs()
    mass = pk.prefill_attention(**a, path=path).float() * (1 + 2.0 ** -6)
    off = (tree.float() - plain.float()).abs()
    assert torch.all(off <= 2 * (2 * 2.0 ** -8 * mass + 2.0 ** -8 * plain.float().abs()))


@pytest.mark.parametrize("path", [1, 3])
def test_errors_in_device_data(path):
    """A sequence with a bad length is left out, a bad parent counts as none, a bad block reads as zeros."""
    pk = require_gpu()
    a = setup(pk)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = pk.tree_attention(**a, path=path, err=err)
    assert err.item() == 0
    b = dict(a, parents=a["parents"].clone())
    b["parents"][3] = 3                      # itself
    b["parents"][9 + 2] = 9                  # beyond its tree
    c = dict(a, parents=b["parents"].clone())
    c["parents"][3] = c["parents"][9 + 2] = -1
    got = pk.tree_attention(**b, path=path, err=err)
    assert err.item() == pk.ERR_TREE
    assert torch.equal(got, pk.tree_attention(**c, path=path))
    err.zero_()
    out = torch.full_like(good, 7.0)
    pk.tree_attention(**dict(a, max_seqlen_q=8), path=path, err=err, out=out)     # the first tree has nine nodes
    assert err.item() == pk.ERR_CONTEXT and torch.all(out[:9] == 7.0) and torch.isfinite(out[9:]).all()
    assert not torch.all(out[9:] == 7.0)
    err.zero_()
    bad = a["cu_seqlens_k"].clone()
    bad[1:] -= 205                           # fewer tokens than drafts
    out.fill_(7.0)
    pk.tree_attention(**dict(a, cu_seqlens_k=bad), path=path, err=err, out=out)
    assert err.item() & pk.ERR_CONTEXT and torch.all(out[:9] == 7.0)
    err.zero_()
    t = a["block_tables"].clone()
    t[0, 2], t[1, 5] = 1 << 30, -7
    out = pk.tree_attention(**dict(a, block_tables=t), path=path, err=err)
    assert err.item() == pk.ERR_BLOCK_ID and torch.isfinite(out).all()


@pytest.mark.parametrize("path", [1, 3])
def test_captured_and_on_other_streams(path):
    """Replays with new data, and two calls at once with workspaces of their own: each bit as when alone."""
    pk = require_gpu()
    a, b = setup(pk, seed=12), setup(pk, seed=13, qlen=(2, 30), cached=(1500, 3))
    ref_a, ref_b = pk.tree_attention(**a, path=path), pk.tree_attention(**b, path=path)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x, y = pk.tree_attention(**a, path=path, stream=s), pk.tree_attention(**b, path=path, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(x, ref_a) and torch.equal(y, ref_b)
    n = pk.tree_workspace_bytes(2, 16, 2, 128, 9)
    ws, out = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(a["q"])
    graph = torch.cuda.CUDAGraph()
    pk.tree_attention(**a, path=path, workspace=ws, out=out)
    with torch.cuda.graph(graph):
        pk.tree_attention(**a, path=path, workspace=ws, out=out)
    q = a["q"].clone()
    a["q"].copy_(torch.randn_like(q))
    graph.replay()
    fresh = out.clone()
    assert torch.equal(fresh, pk.tree_attention(**a, path=path)) and not torch.equal(fresh, ref_a)
    a["q"].copy_(q)
    ws.fill_(0xff)
    graph.replay()
    assert torch.equal(out, ref_a)


def test_blocks_past_32_bit_offsets():
    pk = require_gpu()
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (bs * hkv * d * 2) + 300              # more than 4 GB of keys
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    near, far = ints([[1, 2, 3]]), ints([[nb - 2, nb - 1, nb - 5]])
    g = torch.Generator(device=DEV).manual_seed(0)
    for t in (near, far):
        g.manual_seed(0)
        kc[t[0].long()], vc[t[0].long()] = (torch.randn(3, bs, hkv, d, device=DEV, generator=g).to(kc.dtype) for _ in range(2))
    q = torch.randn(4, 16, d, device=DEV, generator=g).to(kc.dtype)
    for path in (1, 3):
        a, b = (pk.tree_attention(q, kc, vc, t, ints([0, 4]), ints([0, 45]), ints([-1, 0, 0, 1]), 4, d ** -0.5, path=path)
                for t in (near, far))
        assert torch.equal(a, b) and a.abs().sum() > 0


def test_caches_of_other_strides():
    """One layer of a cache of several, K and V side by side; heads before tokens goes to the fp32 path."""
    pk = require_gpu()
    a = setup(pk, hkv=2, hq=8)
    ref = pk.tree_attention(**a)
    nb = a["k_cache"].shape[0]
    both = torch.full((nb, 3, 16, 2, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    both[:, 1, :, 0], both[:, 1, :, 1] = a["k_cache"], a["v_cache"]
    assert torch.equal(pk.tree_attention(**dict(a, k_cache=both[:, 1, :, 0], v_cache=both[:, 1, :, 1])), ref)
    turned = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (a["k_cache"], a["v_cache"])]
    got = pk.tree_attention(**dict(a, k_cache=turned[0], v_cache=turned[1]))
    assert torch.equal(got, pk.tree_attention(**a, path=pk.PATH_FMA))


def test_random_shapes():
    pk = require_gpu()
    rng = np.random.default_rng(2024)
    for seed in range(40):
        d = int(rng.choice([64, 128]))
        hkv = int(rng.choice([1, 2, 3, 8]))
        group = int(rng.choice([1, 2, 3, 5, 8, 12, 33]))
        dt, path = ("f32", 1) if rng.random() < 0.2 else (str(rng.choice(["f16", "bf16"])), int(rng.choice([0, 1, 3])))
        bs = int(rng.choice([16, 32, 128, 256]))
        n = int(rng.integers(1, 8))
        qlen = rng.integers(0, int(rng.choice([3, 20, 90])), n).tolist()
        if max(qlen) == 0:
            qlen[0] = 1
        cached = rng.integers(0, int(rng.choice([20, 400, 2000])), n).tolist()
        mod = (float(rng.choice([0.0, 8.0])), [None, "mixed", "geometric"][int(rng.integers(3))],
               int(rng.choice([0, 0, 1, 50, 200])))
        run_tree(pk, (dt, hkv * group, hkv, d, bs, path), qlen, cached, mod, seed=seed, every=max(1, sum(qlen) * hkv * group // 150))


# ------------------------------------------------------------------- accept
@pytest.mark.parametrize("max_path", [1, 3, 300])
def test_accept(max_path):
    pk = require_gpu()
    rng = np.random.default_rng(max_path)
    qlen = [1, 0, 5, 256, 33, 64, 2] + rng.integers(1, 40, 200).tolist()
    cached = rng.integers(0, 1000, len(qlen)).tolist()
    trees = [a_tree(n, KINDS[i % 4], rng) for i, n in enumerate(qlen)]
    drafted = [rng.integers(0, 3, n) for n in qlen]
    target = [rng.integers(0, 3, n) for n in qlen]
    flat = lambda x: ints([int(v) for row in x for v in row] + [0, 0])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    klen = [c + n for c, n in zip(cached, qlen)]
    pos, first, counts, tokens = pk.tree_accept(flat(drafted), flat(trees), flat(target), cumulative(qlen),
                                                cumulative(klen), max_path, err=err)
    assert err.item() == 0
    longest = 0
    for i, n in enumerate(qlen):
        path = oracle.drafts.accept(drafted[i], trees[i], target[i], max_path)
        longest = max(longest, len(path))
        assert counts[i].item() == len(path) and first[i].item() == cached[i]
        assert pos[i].tolist() == [cached[i] + u for u in path] + [-1] * (max_path - len(path))
        assert tokens[i].tolist() == [int(target[i][u]) for u in path] + [-1] * (max_path - len(path))
    assert longest == min(max_path, longest) and (max_path < 300 or longest > 4)


def test_accept_errors_in_device_data():
    pk = require_gpu()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = ints([0] * 300)
    args = lambda par, cq, ck: (one, par, one, ints(cq), ints(ck), 4)
    pos, first, counts, tokens = pk.tree_accept(*args(ints([-1, 0, 2] + [0] * 297), [0, 3, 3], [0, 3, 3]), err=err)
    assert err.item() == pk.ERR_TREE and counts.tolist() == [2, 0] and pos[0].tolist() == [0, 1, -1, -1]
    err.zero_()
    pos, first, counts, tokens = pk.tree_accept(*args(one - 1, [0, 257], [0, 257]), err=err)      # too many nodes
    assert err.item() == pk.ERR_CONTEXT and counts.tolist() == [0] and torch.all(pos == -1) and torch.all(tokens == -1)
    err.zero_()
    _, _, counts, _ = pk.tree_accept(*args(one - 1, [0, 3, 301], [0, 3, 301]), err=err)           # past the rows
    assert err.item() == pk.ERR_CONTEXT and counts.tolist() == [1, 0]


@pytest.mark.parametrize("case", [("bf16", 48, 8, 128, 16, 3), ("f16", 4, 2, 64, 64, 3), ("bf16", 64, 2, 128, 16, 3),
                                  ("f16", 80, 2, 64, 16, 3), ("bf16", 8, 2, 64, 16, 1), ("f32", 4, 2, 128, 16, 1)],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("window", [0, 20])
def test_values_that_are_no_numbers(case, window):
    """A NaN or an infinity in the V row of a draft, or of a token that a window has left behind for some, reaches
    the nodes that see it in its own column alone, and no other node at all; in K, a draft nobody else sees."""
    pk = require_gpu()
    dt, hq, hkv, d, bs, path = case
    dt, G = DT[dt], hq // hkv
    rng = np.random.default_rng(11)
    qlen, cached = [9, 5, 40, 1, 20], [300, 0, 121, 64, 700]
    klen = [c + n for c, n in zip(cached, qlen)]
    kc, vc, tables, _ = cache_of(klen, hkv, d, bs, dt, 12)
    trees = [a_tree(n, k, rng) for n, k in zip(qlen, ["tree", "star", "forest", "tree", "chain"])]
    q = torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(13)).to(dt).to(DEV)

    def go(k, v):
        return pk.tree_attention(q, k, v, tables, cumulative(qlen), cumulative(klen), ints([u for t in trees for u in t]),
                                 max(qlen), d ** -0.5, window=window, path=path)

    plain = go(kc, vc).float()
    want, k2, v2 = plain.clone(), kc.clone(), vc.clone()
    host = tables.cpu()
    first = np.cumsum([0] + qlen)

    def positions(i):                       # keys that node j sees
        for j in range(qlen[i]):
            up = oracle.drafts.path_of(trees[i], j)
            pos = cached[i] + len(up) - 1
            keys = [(c, c) for c in range(cached[i])] + [(cached[i] + u, cached[i] + n) for n, u in enumerate(up)]
            yield j, {key for key, at in keys if not window or at > pos - window}

    for i in range(len(qlen)):
        sees = dict(positions(i))
        for n, bad in enumerate([float("inf"), float("nan"), float("-inf"), float("inf")]):
            key = cached[i] + int(rng.integers(0, qlen[i])) if n < 3 or not window else max(0, cached[i] - window + 4)
            hk, col = int(rng.integers(0, hkv)), int(rng.integers(0, d))
            v2[host[i, key // bs], key % bs, hk, col] = bad
            for j, seen in sees.items():
                if key in seen:
                    want[first[i] + j, hk * G:(hk + 1) * G, col] += bad
        leaf = qlen[i] - 1                  # the last node: nobody's ancestor
        key = cached[i] + leaf
        k2[host[i, key // bs], key % bs, 0, 3] = float("nan")
        want[first[i] + leaf, :G] = float("nan")
    assert torch.equal(plain.isfinite().all(), torch.tensor(True, device=DEV)) and not want.isfinite().all()
    got = go(k2, v2).float()
    number = want.isfinite()
    assert torch.equal(got[number], plain[number])
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~want.isnan()], want[~want.isnan()])
