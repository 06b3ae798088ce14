"""Operators that change what a paged cache holds, with the work they are measured on.

Two families, each in its plain form (elementary torch operations in 32 bits) and through the library:

* trees of drafted tokens: ``tree_attention`` of every drafted row over its sequence's cache and its ancestors,
  ``tree_accept`` (the path that the target's own choices follow) and ``compact_cache`` (the path's rows move to where
  the sequence goes on);
* eviction by accumulated attention weight: ``paged_decode_attention_weights`` (decode attention that adds up what each
  key was given), ``evict_select`` (the positions that stay) and ``compact_cache`` again (their rows close up).

A case is a dict of plain values; lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a hand-sized draft: four short sequences, a few nodes each, where only the launch counts
        dict(name="tree_tiny", kind="tree", dtype="f32", seqs=4, nlo=1, nhi=6, hq=4, hkv=2, d=64, bs=16, lo=1, hi=50,
             softcap=0.0, alibi=False, window=0),
        # a static batch (48:8 heads, 2048 cached tokens a row) that verifies eight drafted tokens a row
        dict(name="tree_batch", kind="tree", dtype="bf16", seqs=32, nlo=8, nhi=8, hq=48, hkv=8, d=128, bs=16, lo=2048,
             hi=2048, softcap=0.0, alibi=False, window=0),
        # wide trees behind fragmented long contexts
        dict(name="tree_long", kind="tree", dtype="bf16", seqs=16, nlo=64, nhi=64, hq=64, hkv=8, d=128, bs=16, lo=512,
             hi=32768, softcap=0.0, alibi=False, window=0),
        # ragged trees with capped scores over a sliding window, as many KV heads as query heads
        dict(name="tree_capped_window", kind="tree", dtype="f16", seqs=24, nlo=3, nhi=33, hq=16, hkv=16, d=64, bs=256,
             lo=700, hi=8192, softcap=30.0, alibi=False, window=1024),
        # which drafted tokens stay: one small request batch, and the largest trees of a large batch
        dict(name="accept_small", kind="accept", trees=4, nlo=1, nhi=8, path=8, vocab=1000, agree=0.7),
        dict(name="accept_large", kind="accept", trees=512, nlo=60, nhi=256, path=32, vocab=151936, agree=0.9),
        # a batch of decode rows stores its drafts and keeps the accepted ones (the rows move a few places)
        dict(name="compact_drafts", kind="commit", dtype="bf16", seqs=256, nlo=4, nhi=16, hkv=8, d=128, bs=16, lo=64,
             hi=400),
        # long contexts cut to 2048 rows a KV head, into fresh blocks
        dict(name="compact_evicted", kind="move", dtype="bf16", seqs=16, hkv=8, d=128, bs=16, lo=4096, hi=16384,
             keep=2048, per_head=True),
        # the smallest decode rows whose keys' weights are counted
        dict(name="weights_tiny", kind="weights", dtype="f32", seqs=4, hq=4, hkv=2, d=64, bs=16, lo=1, hi=50,
             softcap=0.0, alibi=False, window=0, per_head=True),
        # fragmented long contexts whose keys' weights are counted
        dict(name="weights_long", kind="weights", dtype="bf16", seqs=64, hq=64, hkv=8, d=128, bs=16, lo=512, hi=32768,
             softcap=0.0, alibi=False, window=0, per_head=True),
        # a few short rows, one list of positions for all heads
        dict(name="select_tiny", kind="select", seqs=4, heads=1, lo=1, hi=50, keep=24, sink=2, recent=8, ties=False),
        # the same long contexts cut to 2048 rows a KV head: the first ones, the newest ones and the heaviest
        dict(name="select_long", kind="select", seqs=64, heads=8, lo=4096, hi=32768, keep=2048, sink=4, recent=256,
             ties=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "accept", "commit", "move", "weights", "weights", "select"])
    if kind == "accept":
        nhi = _log_int(rng, 1, 256)
        return dict(kind=kind, trees=_log_int(rng, 1, 512), nlo=max(1, nhi // rng.choice([1, 4])), nhi=nhi,
                    path=_log_int(rng, 1, 64), vocab=_log_int(rng, 2, 152000), agree=rng.choice([0.0, 0.5, 0.9, 1.0]))
    if kind == "select":
        hi = _log_int(rng, 8, 32768)
        keep = _log_int(rng, 1, hi)
        sink = rng.choice([0, min(4, keep)])
        return dict(kind=kind, seqs=_log_int(rng, 1, 64), heads=rng.choice([1, 2, 4, 8]),
                    lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi, keep=keep, sink=sink,
                    recent=rng.choice([0, (keep - sink) // 4, keep - sink]), ties=rng.random() < 0.5)
    d, bs, dtype = rng.choice([64, 128]), rng.choice([16, 32, 64, 256]), rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    if kind in ("commit", "move"):
        dtype = rng.choice(["f32", "f16", "bf16"])
        hi = _log_int(rng, 16, 4096)
        common = dict(kind=kind, dtype=dtype, seqs=_log_int(rng, 1, 48), hkv=hkv, d=d, bs=bs,
                      lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi)
        if kind == "move":
            return dict(common, keep=_log_int(rng, 1, hi), per_head=rng.random() < 0.6)
        nhi = _log_int(rng, 1, 64)
        return dict(common, nlo=max(1, nhi // 4), nhi=nhi)
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    common = dict(kind=kind, dtype=dtype, bs=bs, softcap=cap, alibi=rng.random() < 0.3,
                  window=rng.choice([0, 0, 0, _log_int(rng, 16, 2048)]))
    if kind == "weights":
        d = 64 if hkv == 16 else d
        hi = _log_int(rng, 8, 8192)
        if hkv < 8 and rng.random() < 0.4:
            common["dtype"] = "f32"
        return dict(common, seqs=_log_int(rng, 1, 48), hq=hkv * rng.choice([1, 2, 3, 4, 6, 8]), hkv=hkv, d=d,
                    lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi, per_head=rng.random() < 0.7)
    hi = _log_int(rng, 8, 8192)
    nhi = _log_int(rng, 1, 100)
    if rng.random() < 0.2:              # the 32-bit cache of a small test model
        common["dtype"], hkv, hi = "f32", min(hkv, 4), min(hi, 600)
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    most = max(1, min(32, 400000000 // (nhi * hi * hq)))          # no more than half of the largest listed one
    return dict(common, seqs=_log_int(rng, 1, most), nlo=max(1, nhi // rng.choice([1, 4])), nhi=nhi, hq=hq, hkv=hkv,
                d=d, lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi)


def _lengths(case, lo, hi, n, salt):
    """n lengths, log-uniform in [lo, hi], the first one hi: they follow from the case alone."""
    r = random.Random("%s %d %d %d %s" % (case["kind"], lo, hi, n, salt))
    return [hi] + [_log_int(r, lo, hi) for _ in range(n - 1)]


def _context_lengths(case):
    return _lengths(case, case["lo"], case["hi"], case["seqs"], "context")


def _node_counts(case):
    return _lengths(case, case["nlo"], case["nhi"], case["trees"] if case["kind"] == "accept" else case["seqs"], "nodes")


def slopes_of(heads):
    """Head h's slope 2^(-8 (h + 1) / heads)."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32)


# ----------------------------------------------------------------- prepare
def _normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=TYPES[dtype], device=DEV).normal_(0.0, std, generator=g)


def _tables(lens, bs, order, at):
    """Block tables for rows of these lengths, their blocks order[at:]; -1 behind each row's last one."""
    need = [-(-n // bs) for n in lens]
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    for i, ids in enumerate(order[at:at + sum(need)].split(need)):
        tables[i, :need[i]] = ids
    return tables, at + sum(need)


def _paged(case, g, lens, fresh=()):
    """A cache of the blocks that the rows need, in a random order over the pool, and their block tables; with `fresh`
    lengths a second set of tables over blocks of its own."""
    bs = case["bs"]
    nb = sum(-(-n // bs) for n in lens) + sum(-(-n // bs) for n in fresh) + 1
    order = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables, at = _tables(lens, bs, order, 0)
    more = _tables(fresh, bs, order, at)[0] if fresh else None
    shape = (nb, bs, case["hkv"], case["d"])
    return tables, more, _normal(g, shape, case["dtype"]), _normal(g, shape, case["dtype"])


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cumulative(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def _parents(g, counts):
    """Trees whose node t hangs on one of the four nodes before it (node 0 on the cache)."""
    local = torch.cat([torch.arange(n, device=DEV) for n in counts])
    back = torch.rand(local.shape[0], generator=g, device=DEV) * local.clamp(max=4)
    return torch.where(local > 0, local - 1 - back.long().clamp(max=3), -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=dict(case))
    kind = case["kind"]
    if kind == "accept":
        counts = _node_counts(case)
        n = sum(counts)
        s["cu_q"] = _cumulative(counts)
        s["cu_k"] = _cumulative([c + 100 + 7 * i for i, c in enumerate(counts)])     # some tokens are cached
        s["parents"] = _parents(g, counts)
        s["target"] = torch.randint(0, case["vocab"], (n,), generator=g, device=DEV, dtype=torch.int32)
        s["drafted"] = torch.randint(0, case["vocab"], (n,), generator=g, device=DEV, dtype=torch.int32)
        # the draft agrees with the target's choice after a node's parent for a share of the nodes
        first = torch.repeat_interleave(s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long())
        after = s["target"][first + s["parents"].long().clamp(min=0)]
        agrees = torch.rand(n, generator=g, device=DEV) < case["agree"]
        s["drafted"] = torch.where(agrees, after, s["drafted"])
        return s
    lens = _context_lengths(case)
    if kind == "select":
        s["ctx"] = _ints(lens)
        w = torch.empty(case["seqs"], case["heads"], case["hi"], device=DEV).exponential_(1.0, generator=g) ** 3
        s["weights"] = torch.round(w * 16) / 16 if case["ties"] else w
        s["weights_out"] = torch.empty_like(w)
        return s
    hkv, d = case["hkv"], case["d"]
    if kind == "move":
        kept = [min(n, case["keep"]) for n in lens]
        s["tables"], s["new_tables"], s["kc"], s["vc"] = _paged(case, g, lens, kept)
        s["counts"] = _ints(kept)
        heads = hkv if case["per_head"] else 1
        score = torch.rand(case["seqs"], heads, case["hi"], generator=g, device=DEV)
        score = score.masked_fill(torch.arange(case["hi"], device=DEV) >= _ints(lens)[:, None, None], -1.0)
        keep = min(case["keep"], case["hi"])
        at = score.topk(keep, dim=2).indices                   # a row with fewer: those behind it sort to the end
        at = at.masked_fill(score.gather(2, at) < 0, case["hi"]).sort(dim=2).values
        s["positions"] = at.masked_fill(at == case["hi"], -1).to(torch.int32)
        if not case["per_head"]:
            s["positions"] = s["positions"][:, 0].contiguous()
        return s
    if kind == "commit":
        counts = _node_counts(case)
        total = [n + c for n, c in zip(lens, counts)]
        s["tables"], _, s["kc"], s["vc"] = _paged(case, g, total)
        s["cu_q"], s["cu_k"], s["first"] = _cumulative(counts), _cumulative(total), _ints(lens)
        s["k"], s["v"] = (_normal(g, (sum(counts), hkv, d), case["dtype"]) for _ in range(2))
        # the accepted rows: node 0 and some of the later ones, as a path through a tree has them
        width = max(counts)
        stays = torch.rand(case["seqs"], width, generator=g, device=DEV) < 0.4
        stays[:, 0] = True
        stays &= torch.arange(width, device=DEV) < _ints(counts)[:, None]
        s["counts"] = stays.sum(dim=1).to(torch.int32)
        at = torch.where(stays, torch.arange(width, device=DEV), width).sort(dim=1).values
        s["positions"] = torch.where(at < width, at + s["first"][:, None], -1).to(torch.int32)
        return s
    # scores of a few units either way, so that a cap of some tens bends the largest ones
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = slopes_of(case["hq"]).to(DEV) if case["alibi"] else None
    if kind == "weights":
        s["ctx"], s["max_ctx"] = _ints(lens), max(lens)
        s["tables"], _, s["kc"], s["vc"] = _paged(case, g, lens)
        s["q"] = _normal(g, (case["seqs"], case["hq"], d), case["dtype"], 3.0)
        # what earlier steps gave the keys
        shape = (case["seqs"], hkv if case["per_head"] else 1, max(lens))
        s["weights"] = torch.empty(shape, device=DEV).exponential_(100.0, generator=g)
        s["weights_out"] = torch.zeros_like(s["weights"])
        if own:      # the scratch that a serving loop keeps
            import paged_kv_decode_store_gb300 as pk
            n = pk.decode_weights_workspace_bytes(case["seqs"], case["hq"], d, max(lens))
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        return s
    counts = _node_counts(case)
    total = [n + c for n, c in zip(lens, counts)]
    s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cumulative(counts), _cumulative(total), max(counts), max(total)
    s["tables"], _, s["kc"], s["vc"] = _paged(case, g, total)
    s["parents"] = _parents(g, counts)
    s["q"] = _normal(g, (sum(counts), case["hq"], d), case["dtype"], 3.0)
    if own:
        import paged_kv_decode_store_gb300 as pk
        n = pk.tree_workspace_bytes(case["seqs"], case["hq"], hkv, d, s["max_q"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- plain forms
def _gathered(s, cache, length):
    """Every row's context side by side, in 32 bits: [rows, Hkv, length, D] (what lies past a context is masked)."""
    x = cache[s["tables"].clamp(min=0).to(torch.int64)].flatten(1, 2)[:, :length]
    return x.float().transpose(1, 2)


def _scored(s, scores, visible, distance):
    """Softmax weights of the capped and biased scores [..., Hkv, G, Q, K] over the visible keys."""
    c = s["case"]
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    if s["slopes"] is not None:
        scores = scores - s["slopes"].view(c["hkv"], -1, 1, 1) * distance
    scores = scores.masked_fill(~visible, float("-inf"))
    weights = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return weights / weights.sum(dim=-1, keepdim=True)


def _ancestors(local, parents, counts, width):
    """[trees, width, width]: which nodes lie on the way from a node to the cache, itself among them; and depths."""
    n = len(counts)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), _ints(counts).long())
    up = torch.full((n, width), -1, dtype=torch.int64, device=DEV)
    up[seq, local] = parents.long()
    own_row = torch.eye(width, dtype=torch.bool, device=DEV).expand(n, -1, -1)
    on_way, at = own_row.clone(), up.clone()
    depth = torch.zeros(n, width, dtype=torch.int64, device=DEV)
    for _ in range(width - 1):
        there = at >= 0
        step = torch.zeros_like(on_way).scatter_(2, at.clamp(min=0)[:, :, None], there[:, :, None])
        on_way |= step
        depth += there
        at = torch.where(there, up.gather(1, at.clamp(min=0)), -1)
    return on_way, depth, seq


def _plain_tree(s):
    c = s["case"]
    n, hkv, hq, d, mk = c["seqs"], c["hkv"], c["hq"], c["d"], s["max_k"]
    counts, lens = _node_counts(c), _context_lengths(c)
    mq = s["max_q"]
    local = torch.cat([torch.arange(m, device=DEV) for m in counts])
    on_way, depth, seq = _ancestors(local, s["parents"], counts, mq)
    q = torch.zeros(n, mq, hq, d, device=DEV)
    q[seq, local] = s["q"].float()
    q = q.view(n, mq, hkv, -1, d).permute(0, 2, 3, 1, 4)        # [n, Hkv, G, Q, D]
    scores = torch.matmul(q.flatten(2, 3), _gathered(s, s["kc"], mk).transpose(2, 3)) * s["scale"]
    cached = _ints(lens).long()[:, None]
    j = torch.arange(mk, device=DEV)
    node = (j - cached).clamp(min=0, max=mq - 1)                # the node that a key past the cache belongs to
    place = torch.where(j < cached, j, cached + depth.gather(1, node))             # every key's position
    back = (cached + depth)[:, :, None] - place[:, None, :]
    held = cached + _ints(counts).long()[:, None]               # tokens of each sequence, its drafts among them
    drafted = on_way.gather(2, node[:, None, :].expand(-1, mq, -1)) & (j < held)[:, None, :]
    visible = torch.where((j < cached)[:, None, :], True, drafted)
    if c["window"]:
        visible = visible & (back < c["window"])
    w = _scored(s, scores.view(n, hkv, -1, mq, mk), visible.view(n, 1, 1, mq, mk),
                back.float().view(n, 1, 1, mq, mk))
    out = torch.matmul(w.flatten(2, 3), _gathered(s, s["vc"], mk))
    out = out.view(n, hkv, -1, mq, d).permute(0, 3, 1, 2, 4).reshape(n, mq, hq, d)
    return out[seq, local].to(s["q"].dtype)


def _plain_weights(s):
    c = s["case"]
    n, hkv, d, mk = c["seqs"], c["hkv"], c["d"], s["max_ctx"]
    q = s["q"].float().view(n, hkv, -1, d)
    scores = torch.matmul(q, _gathered(s, s["kc"], mk).transpose(2, 3)) * s["scale"]
    back = s["ctx"].to(torch.int64)[:, None] - 1 - torch.arange(mk, device=DEV)   # how far a key lies behind
    visible = back >= 0
    if c["window"]:
        visible = visible & (back < c["window"])
    w = _scored(s, scores.unsqueeze(3), visible.view(n, 1, 1, 1, -1), back.float().view(n, 1, 1, 1, -1)).squeeze(3)
    out = torch.matmul(w, _gathered(s, s["vc"], mk)).reshape(n, -1, d).to(s["q"].dtype)
    given = w.sum(dim=2)
    if not c["per_head"]:
        given = given.sum(dim=1, keepdim=True)
    s["weights_out"].copy_(torch.where((back >= 0)[:, None], s["weights"] + given, s["weights_out"]))
    return out, s["weights_out"]


def _plain_accept(s):
    """All trees one step at a time."""
    c = s["case"]
    n, width = c["trees"], c["path"]
    first, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    cached = (s["cu_k"][1:] - s["cu_k"][:-1]).long() - count
    m = c["nhi"]
    j = torch.arange(m, device=DEV)
    at = (first[:, None] + j).clamp(max=s["parents"].shape[0] - 1)
    real = j < count[:, None]
    up, drafted = s["parents"][at].long(), s["drafted"][at]
    here = torch.zeros(n, dtype=torch.int64, device=DEV)
    alive = count > 0
    positions = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    tokens = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    length = torch.zeros(n, dtype=torch.int32, device=DEV)
    for step in range(min(width, m)):
        choice = s["target"][first + here]
        positions[:, step] = torch.where(alive, cached + here, -1).to(torch.int32)
        tokens[:, step] = torch.where(alive, choice, -1)
        length += alive
        follows = real & (up == here[:, None]) & (j > here[:, None]) & (drafted == choice[:, None])
        alive = alive & follows.any(dim=1)
        here = torch.where(alive, follows.to(torch.int8).argmax(dim=1), here)
    return positions, cached.to(torch.int32), length, tokens


def _moved(s, cache, tables, positions, counts, first, new_tables):
    """The cache with row first + r of every new table set to row positions[r] of the table, head by head."""
    c = s["case"]
    hkv, bs = c["hkv"], c["bs"]
    if positions.dim() == 2:
        positions = positions[:, None].expand(-1, hkv, -1)
    seq, head, r = torch.nonzero(torch.arange(positions.shape[2], device=DEV) < counts[:, None, None].expand(
        -1, hkv, -1), as_tuple=True)
    src, dst = positions[seq, head, r].long(), r + first[seq].long()
    rows = cache[tables[seq, src // bs].long(), src % bs, head]
    cache[new_tables[seq, dst // bs].long(), dst % bs, head] = rows


def _plain_commit(s):
    bs = s["case"]["bs"]
    rows = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(s["cu_q"][1:].to(torch.int64), rows, right=True)
    pos = s["first"].long()[seq] + rows - s["cu_q"].long()[seq]
    block = s["tables"][seq, pos // bs].long()
    for cache, new in ((s["kc"], s["k"]), (s["vc"], s["v"])):
        cache[block, pos % bs] = new
        _moved(s, cache, s["tables"], s["positions"], s["counts"], s["first"], s["tables"])
    return s["kc"], s["vc"]


def _plain_move(s):
    for cache in (s["kc"], s["vc"]):
        _moved(s, cache, s["tables"], s["positions"], s["counts"], torch.zeros_like(s["counts"]), s["new_tables"])
    return s["kc"], s["vc"]


def _plain_select(s):
    c = s["case"]
    w, n, keep = s["weights"], c["hi"], c["keep"]
    ctx = s["ctx"].long()[:, None, None]
    j = torch.arange(n, device=DEV)
    always = (j < c["sink"]) | (j >= ctx - c["recent"])
    rank = torch.where(always, float("inf"), w)
    rank = torch.where(j < ctx, rank, float("-inf"))
    at = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    if at.shape[2] < keep:
        at = torch.nn.functional.pad(at, (0, keep - at.shape[2]), value=n)
    counts = s["ctx"].clamp(max=keep)
    at = torch.where(torch.arange(keep, device=DEV) < counts[:, None, None], at, n).sort(dim=2).values
    held = torch.nn.functional.pad(w, (0, 1)).gather(2, at)
    s["weights_out"].zero_()
    m = min(keep, n)
    s["weights_out"][:, :, :m] = held[:, :, :m]
    return torch.where(at < n, at, -1).to(torch.int32), counts, s["weights_out"]


# --------------------------------------------------------------------- run
def _own(s):
    import paged_kv_decode_store_gb300 as pk
    c = s["case"]
    kind = c["kind"]
    if kind == "tree":
        return pk.tree_attention(s["q"], s["kc"], s["vc"], s["tables"], s["cu_q"], s["cu_k"], s["parents"], s["max_q"],
                                 s["scale"], window=c["window"], softcap=c["softcap"], alibi_slopes=s["slopes"],
                                 workspace=s["workspace"])
    if kind == "accept":
        return pk.tree_accept(s["drafted"], s["parents"], s["target"], s["cu_q"], s["cu_k"], c["path"])
    if kind == "commit":
        pk.kv_store_prefill(s["k"], s["v"], s["tables"], s["cu_q"], s["cu_k"], s["kc"], s["vc"])
        pk.compact_cache(s["kc"], s["vc"], s["tables"], s["positions"], s["counts"], first=s["first"])
        return s["kc"], s["vc"]
    if kind == "move":
        pk.compact_cache(s["kc"], s["vc"], s["tables"], s["positions"], s["counts"], new_tables=s["new_tables"])
        return s["kc"], s["vc"]
    if kind == "weights":
        return pk.paged_decode_attention_weights(s["q"], s["kc"], s["vc"], s["tables"], s["ctx"], s["max_ctx"],
                                                 s["scale"], s["weights"], weights_out=s["weights_out"],
                                                 workspace=s["workspace"], window=c["window"], softcap=c["softcap"],
                                                 alibi_slopes=s["slopes"])
    positions, counts = pk.evict_select(s["weights"], s["ctx"], c["keep"], sink=c["sink"], recent=c["recent"],
                                        weights_out=s["weights_out"])
    return positions, counts, s["weights_out"]


PLAIN = {"tree": _plain_tree, "accept": _plain_accept, "commit": _plain_commit, "move": _plain_move,
         "weights": _plain_weights, "select": _plain_select}


def run(s):
    return _own(s) if own else PLAIN[s["case"]["kind"]](s)


# -------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    if kind == "accept":
        n = sum(_node_counts(case))
        return {"bytes": 12 * n + case["trees"] * (16 + 8 * case["path"]), "flops": 2 * n}
    lens = _context_lengths(case)
    if kind == "select":
        rows = case["seqs"] * case["heads"]
        n = sum(lens) * case["heads"]
        return {"bytes": 4 * n + 4 * rows * (case["keep"] + case["hi"]) + 8 * case["seqs"], "flops": n}
    e = SIZE[case["dtype"]]
    hkv, d = case["hkv"], case["d"]
    if kind == "move":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": 4 * kept * hkv * d * e + 4 * kept * (hkv if case["per_head"] else 1), "flops": 0}
    counts = _node_counts(case) if "nlo" in case else []
    if kind == "commit":
        t = sum(counts)
        return {"bytes": 4 * t * hkv * d * e + 4 * t, "flops": 0}
    hq, window = case["hq"], case["window"]
    if kind == "weights":
        seen = sum(min(n, window) if window else n for n in lens)
        heads = hkv if case["per_head"] else 1
        return {"bytes": 2 * seen * hkv * d * e + 2 * len(lens) * hq * d * e + 8 * sum(lens) * heads,
                "flops": 4 * seen * hq * d}
    # a node's ancestors depend on the seed: at least itself
    read = [m + (min(n, window) if window else n) for n, m in zip(lens, counts)]
    pairs = sum(m * ((min(n, window - 1) if window else n) + 1) for n, m in zip(lens, counts))
    return {"bytes": 2 * sum(read) * hkv * d * e + 2 * sum(counts) * hq * d * e, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact
def _softmax64(s, x, seen, distance, heads):
    """Weights in 64 bits of raw products x [G, rows, keys] of the query heads `heads`."""
    c = s["case"]
    x = x * s["scale"]
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    if s["slopes"] is not None:
        x = x - s["slopes"][heads].double()[:, None, None] * distance
    return torch.softmax(torch.where(seen, x, torch.full_like(x, -math.inf)), dim=-1)


def _rows64(s, i, n):
    c = s["case"]
    ids = s["tables"][i, :-(-n // c["bs"])].to(torch.int64)
    return [x[ids].reshape(-1, c["hkv"], c["d"])[:n].double() for x in (s["kc"], s["vc"])]


def _exact_tree(s):
    """One sequence, and one KV head of it, at a time; a node's ancestors by walking up."""
    c = s["case"]
    hkv, group = c["hkv"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    a = 0
    for i, (n, m) in enumerate(zip(_context_lengths(c), _node_counts(c))):
        up = s["parents"][a:a + m].tolist()
        way = [[t] for t in range(m)]
        for t in range(m):
            if up[t] >= 0:
                way[t] = way[up[t]] + [t]
        depth = torch.tensor([len(w) - 1 for w in way], device=DEV)
        tree = torch.zeros(m, m, dtype=torch.bool)
        for t in range(m):
            tree[t, way[t]] = True
        seen = torch.cat((torch.ones(m, n, dtype=torch.bool, device=DEV), tree.to(DEV)), dim=1)
        distance = (n + depth)[:, None] - torch.cat((torch.arange(n, device=DEV), n + depth))[None]
        if c["window"]:
            seen = seen & (distance < c["window"])
        key, val = _rows64(s, i, n + m)
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            x = torch.einsum("rgd,nd->grn", s["q"][a:a + m, heads].double(), key[:, h])
            out[a:a + m, heads] = torch.einsum("grn,nd->rgd", _softmax64(s, x, seen, distance, heads), val[:, h])
        a += m
    return out


def _exact_weights(s):
    c = s["case"]
    hkv, group = c["hkv"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    total = s["weights_out"].double()
    for i, n in enumerate(_context_lengths(c)):
        key, val = _rows64(s, i, n)
        distance = torch.arange(n - 1, -1, -1, device=DEV)[None]
        seen = distance < c["window"] if c["window"] else distance >= 0
        total[i, :, :n] = s["weights"][i, :, :n].double()
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            x = torch.einsum("gd,nd->gn", s["q"][i, heads].double(), key[:, h])[:, None]
            w = _softmax64(s, x, seen, distance, heads)[:, 0]
            out[i, heads] = w @ val[:, h]
            total[i, h if c["per_head"] else 0, :n] += w.sum(dim=0)
    return out, total


def _slots(table, positions, bs):
    return table[positions // bs].long() * bs + positions % bs


def _exact_rows(s):
    """Sequence by sequence and head by head, over the caches as lists of rows."""
    c = s["case"]
    hkv, bs = c["hkv"], c["bs"]
    caches = [x.double().view(-1, hkv, c["d"]) for x in (s["kc"], s["vc"])]
    old, new, counts = s["tables"], s.get("new_tables", s["tables"]), s["counts"].tolist()
    for i, n in enumerate(counts):
        start = int(s["first"][i]) if "first" in s else 0
        if c["kind"] == "commit":
            a, b = s["cu_q"][i:i + 2].tolist()
            at = _slots(old[i], torch.arange(start, start + b - a, device=DEV), bs)
            caches[0][at], caches[1][at] = s["k"][a:b].double(), s["v"][a:b].double()
        to = _slots(new[i], torch.arange(start, start + n, device=DEV), bs)
        for h in range(hkv):
            keep = s["positions"][i] if s["positions"].dim() == 2 else s["positions"][i, h]
            at = _slots(old[i], keep[:n].long(), bs)
            for x in caches:
                x[to, h] = x[at, h].clone()
    return tuple(x.view(s["kc"].shape) for x in caches)


def _exact_select(s):
    """The weights that stay, row by row; positions and counts are whole numbers."""
    c = s["case"]
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_context_lengths(c)):
        for h in range(c["heads"]):
            w = s["weights"][i, h, :n].double()
            if n > c["keep"]:
                m = n - c["recent"]
                middle = w[c["sink"]:m]
                order = torch.argsort(middle, descending=True, stable=True)
                stay = order[:c["keep"] - c["sink"] - c["recent"]].sort().values
                w = torch.cat((w[:c["sink"]], middle[stay], w[m:]))
            out[i, h, :w.shape[0]] = w
    return None, None, out


def exact(case, seed):
    if case["kind"] == "accept":
        return None                    # whole numbers
    s = prepare(case, seed)
    return {"tree": _exact_tree, "weights": _exact_weights, "commit": _exact_rows, "move": _exact_rows,
            "select": _exact_select}[case["kind"]](s)
