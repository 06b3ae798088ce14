"""Operators around the paged decode step, with the work they are measured on.

Three families, each in its plain form (elementary torch operations in 32 or 64 bits) and through the library:

* rotary positions: ``rope`` on projected rows, and fused with the paged store of a decode step
  (``rope_store_paged``) or of a varlen prefill batch (``rope_store_prefill``);
* attention over the paged cache whose scores are capped by a tanh, biased by distance or opened to a
  bidirectional prefix: ``paged_decode_attention`` and ``prefill_attention`` with ``softcap``,
  ``alibi_slopes`` and ``prefix_lens``;
* one step of beam search: ``beam_search_step`` over beams and vocabulary.

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
        # a hand-sized decode step: four rows, where only the launch counts
        dict(name="rope_store_tiny", kind="rope_decode", dtype="f32", seqs=4, hq=4, hkv=2, d=64, bs=16, lo=1, hi=50,
             rot=64, interleaved=False, scaling="none"),
        # the decode step of a full long-context batch
        dict(name="rope_store_batch", kind="rope_decode", dtype="bf16", seqs=256, hq=64, hkv=8, d=128, bs=16, lo=512,
             hi=8192, rot=128, interleaved=False, scaling="linear"),
        # eight prompts padded to 1024 tokens, 48 query heads over 8 KV heads
        dict(name="rope_store_prefill", kind="rope_prefill", dtype="bf16", seqs=8, hq=48, hkv=8, d=128, bs=16,
             qlo=1024, qhi=1024, cached=0, rot=128, interleaved=True, scaling="none"),
        # ragged prompts at far positions of a stretched context, half of each head rotated, read from fused QKV rows
        dict(name="rope_far_partial", kind="rope", dtype="f16", tokens=18433, hq=16, hkv=16, d=64, far=1 << 20, rot=32,
             interleaved=False, scaling="parts"),
        # the smallest decode call: rows of 1 to 50 tokens, cap and distance bias together
        dict(name="decode_tiny", kind="decode", dtype="f32", seqs=4, hq=4, hkv=2, d=64, bs=16, lo=1, hi=50,
             softcap=20.0, alibi=True, window=0),
        # a static padded batch with capped scores (48:8 heads, 2048 tokens a row)
        dict(name="decode_capped", kind="decode", dtype="bf16", seqs=32, hq=48, hkv=8, d=128, bs=16, lo=2048, hi=2048,
             softcap=30.0, alibi=False, window=0),
        # fragmented long contexts with a distance bias
        dict(name="decode_biased_long", kind="decode", dtype="bf16", seqs=64, hq=64, hkv=8, d=128, bs=16, lo=512,
             hi=32768, softcap=0.0, alibi=True, window=0),
        # eight prompts of 1024 tokens with capped scores
        dict(name="prefill_capped", kind="prefill", dtype="bf16", seqs=8, hq=48, hkv=8, d=128, bs=16, qlo=1024,
             qhi=1024, cached=0, softcap=30.0, alibi=False, prefix=0, window=0),
        # chunks of 1024 tokens after up to seven earlier ones: distance bias, and prompts read in both directions
        dict(name="prefill_prefix_chunk", kind="prefill", dtype="f16", seqs=4, hq=64, hkv=8, d=64, bs=256, qlo=900,
             qhi=1024, cached=7168, softcap=0.0, alibi=True, prefix=2500, window=0),
        # beam search of one request over a small vocabulary
        dict(name="beam_tiny", kind="beam", dtype="f32", reqs=1, beams=4, vocab=1000, keep=4, done=False),
        # sixteen requests of four beams, twice as many continuations kept, some beams ended
        dict(name="beam_batch", kind="beam", dtype="bf16", reqs=16, beams=4, vocab=65536, keep=8, done=True),
        # the largest: 64 requests of eight beams over 151,936 ids
        dict(name="beam_large", kind="beam", dtype="f16", reqs=64, beams=8, vocab=151936, keep=16, done=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope_decode", "rope_prefill", "decode", "prefill", "beam"])
    d = rng.choice([64, 128])
    bs = rng.choice([16, 32, 64, 256])
    if kind == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8])
        return dict(kind=kind, dtype=rng.choice(["f32", "f16", "bf16"]), reqs=_log_int(rng, 1, 32), beams=beams,
                    vocab=_log_int(rng, 500, 152000), keep=rng.choice([1, beams, 2 * beams]), done=rng.random() < 0.4)
    if kind == "decode":
        hkv = rng.choice([1, 2, 4, 8, 8, 16])
        d = 64 if hkv == 16 else d
        hi = _log_int(rng, 16, 8192)
        cap = rng.choice([0.0, 20.0, 30.0, 50.0])
        return dict(kind=kind, dtype=rng.choice(["f16", "bf16", "bf16", "f32"] if hkv < 8 else ["f16", "bf16"]),
                    seqs=_log_int(rng, 1, 48), hq=hkv * rng.choice([1, 2, 3, 4, 6, 8]), hkv=hkv, d=d, bs=bs,
                    lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi, softcap=cap, alibi=cap == 0.0 or rng.random() < 0.5,
                    window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]))
    if kind == "prefill":
        hkv = rng.choice([1, 2, 4, 8])
        qhi = _log_int(rng, 8, 768)
        cap = rng.choice([0.0, 20.0, 30.0, 50.0])
        return dict(kind=kind, dtype=rng.choice(["f16", "bf16"]), seqs=rng.randint(1, 4),
                    hq=hkv * rng.choice([1, 2, 4, 6]), hkv=hkv, d=d, bs=bs, qlo=max(1, qhi // rng.choice([1, 2, 8])),
                    qhi=qhi, cached=rng.choice([0, 0, _log_int(rng, 16, 2048)]), softcap=cap,
                    alibi=cap == 0.0 or rng.random() < 0.5, prefix=rng.choice([0, 0, _log_int(rng, 8, 2048)]),
                    window=rng.choice([0, 0, 0, _log_int(rng, 16, 1024)]))
    hkv = rng.choice([1, 2, 4, 8, 16])
    common = dict(kind=kind, dtype=rng.choice(["f32", "f16", "bf16"]), hq=hkv * rng.choice([1, 2, 3, 4]), hkv=hkv, d=d,
                  rot=rng.choice([d, d // 2, d // 4, d - 16]), interleaved=rng.random() < 0.5,
                  scaling=rng.choice(["none", "linear", "ntk", "parts"]))
    if kind == "rope":
        return dict(common, tokens=_log_int(rng, 1, 4096), far=_log_int(rng, 64, 1 << 22))
    if kind == "rope_decode":
        hi = _log_int(rng, 4, 4096)
        return dict(common, seqs=_log_int(rng, 1, 256), bs=bs, lo=max(1, hi // 8), hi=hi)
    qhi = _log_int(rng, 4, 1024)
    return dict(common, seqs=rng.randint(1, 8), bs=bs, qlo=max(1, qhi // rng.choice([1, 4])), qhi=qhi,
                cached=rng.choice([0, _log_int(rng, 16, 2048)]))


def _lengths(case, lo, hi, n, salt):
    """n lengths, log-uniform in [lo, hi], the first one hi: they follow from the case alone."""
    r = random.Random("%s %d %d %d %s" % (case["kind"], lo, hi, n, salt))
    return [hi] + [_log_int(r, lo, hi) for _ in range(n - 1)]


def _query_lengths(case):
    return _lengths(case, case["qlo"], case["qhi"], case["seqs"], "q")


def _cached_lengths(case):
    """Tokens already in the cache, any number of them up to the case's."""
    r = random.Random("%d %d %d" % (case["cached"], case["seqs"], case["qhi"]))
    return [case["cached"]] + [r.randint(0, case["cached"]) for _ in range(case["seqs"] - 1)]


def _prefix_lengths(case, klens):
    r = random.Random("%d %d" % (case["prefix"], case["seqs"]))
    return [min(k, case["prefix"] if i == 0 else r.randint(0, case["prefix"])) for i, k in enumerate(klens)]


def inv_freq_of(case):
    """(inverse frequencies, factor on cos and sin) of a head's rotated part, in 64 bits: plain, positions divided by
    the stretch, a larger base, or by parts (low frequencies stretched, high ones kept, a ramp between)."""
    rot, base, stretch, original = case["rot"], 10000.0, 8.0, 4096.0
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * stretch ** (rot / (rot - 2)) if rot > 2 else base
    inv = base ** (-i / rot)
    if case["scaling"] == "linear":
        return inv / stretch, 1.0
    if case["scaling"] == "parts":
        def pair_of(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        return inv * (1 - ramp) + inv / stretch * ramp, 0.1 * math.log(stretch) + 1.0
    return inv, 1.0


def slopes_of(heads):
    """Head h's slope 2^(-8 (h + 1) / heads)."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32)


# ----------------------------------------------------------------- prepare
def _normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=TYPES[dtype], device=DEV).normal_(0.0, std, generator=g)


def _paged(case, g, lens):
    """A cache of the blocks that the rows need, in a random order over the pool, and their block tables."""
    bs = case["bs"]
    need = [-(-n // bs) for n in lens]
    nb, width = sum(need) + 1, max(need)
    order = torch.randperm(nb, generator=g, device=DEV)[:sum(need)].to(torch.int32).split(need)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    for i, ids in enumerate(order):
        tables[i, :need[i]] = ids
    shape = (nb, bs, case["hkv"], case["d"])
    return tables, _normal(g, shape, case["dtype"]), _normal(g, shape, case["dtype"])


def _cumulative(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=dict(case))
    if case["kind"] == "beam":
        n, b, v = case["reqs"], case["beams"], case["vocab"]
        s["logits"] = _normal(g, (n * b, v), case["dtype"], 3.0)
        s["scores"] = -torch.empty(n, b, device=DEV).exponential_(0.2, generator=g).sort(dim=1)[0]
        s["finished"] = None
        if case["done"]:      # about a quarter of the beams have ended; id 2 ends a beam
            s["finished"] = (torch.rand(n, b, generator=g, device=DEV) < 0.25).to(torch.uint8)
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["kind"].startswith("rope"):
        inv, s["mscale"] = inv_freq_of(case)
        s["inv_freq"] = inv.to(DEV)
        if case["kind"] == "rope":
            t = case["tokens"]
            # the projection's output: Q, K and V of a token side by side
            qkv = _normal(g, (t, hq + 2 * hkv, d), case["dtype"])
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
            s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV)
            return s
        if case["kind"] == "rope_decode":
            lens = _lengths(case, case["lo"], case["hi"], case["seqs"], "ctx")
            t = case["seqs"]
            s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        else:
            qlens = _query_lengths(case)
            lens = [q + c for q, c in zip(qlens, _cached_lengths(case))]
            t = sum(qlens)
            s["cu_q"], s["cu_k"] = _cumulative(qlens), _cumulative(lens)
        s["tables"], s["kc"], s["vc"] = _paged(case, g, lens)
        qkv = _normal(g, (t, hq + 2 * hkv, d), case["dtype"])
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        return s
    # scores of a few units either way, so that a cap of some tens bends the largest ones
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = slopes_of(hq).to(DEV) if case["alibi"] else None
    if case["kind"] == "decode":
        lens = _lengths(case, case["lo"], case["hi"], case["seqs"], "ctx")
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["max_ctx"] = max(lens)
        s["tables"], s["kc"], s["vc"] = _paged(case, g, lens)
        s["q"] = _normal(g, (case["seqs"], hq, d), case["dtype"], 3.0)
        # the scratch that a serving loop keeps: enough for every head layout on this GPU
        s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
        return s
    qlens = _query_lengths(case)
    lens = [q + c for q, c in zip(qlens, _cached_lengths(case))]
    s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cumulative(qlens), _cumulative(lens), max(qlens), max(lens)
    s["prefix"] = None
    if case["prefix"]:
        s["prefix"] = torch.tensor(_prefix_lengths(case, lens), dtype=torch.int32, device=DEV)
    s["tables"], s["kc"], s["vc"] = _paged(case, g, lens)
    s["q"] = _normal(g, (sum(qlens), hq, d), case["dtype"], 3.0)
    return s


# -------------------------------------------------------------- plain forms
def _rotated(x, positions, inv_freq, interleaved, mscale):
    """x [T, H, D] in 32 bits with the first 2 len(inv_freq) dims of every head rotated by position * inv_freq;
    the angles, their cos and sin in 64 bits."""
    angle = positions.to(torch.float64)[:, None] * inv_freq
    cos = (torch.cos(angle) * mscale).float()[:, None]
    sin = (torch.sin(angle) * mscale).float()[:, None]
    x = x.float()
    r = 2 * inv_freq.shape[0]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., r:]), dim=-1)


def _rows_of(cu_q, cu_k, total):
    """Each new row's sequence and position in it."""
    rows = torch.arange(total, device=cu_q.device)
    seq = torch.searchsorted(cu_q[1:].to(torch.int64), rows, right=True)
    qlen, klen = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    return seq, (klen - qlen)[seq] + rows - cu_q[seq]


def _plain_rope(s):
    c = s["case"]
    turn = (s["inv_freq"], c["interleaved"], s["mscale"])
    dt = s["q"].dtype
    if c["kind"] == "rope":
        return _rotated(s["q"], s["positions"], *turn).to(dt), _rotated(s["k"], s["positions"], *turn).to(dt)
    if c["kind"] == "rope_decode":
        pos = s["ctx"].to(torch.int64) - 1
        seq = torch.arange(pos.shape[0], device=pos.device)
    else:
        seq, pos = _rows_of(s["cu_q"], s["cu_k"], s["q"].shape[0])
    slots = s["tables"][seq, pos // c["bs"]].to(torch.int64) * c["bs"] + pos % c["bs"]
    q = _rotated(s["q"], pos, *turn).to(dt)
    s["kc"].view(-1, c["hkv"], c["d"])[slots] = _rotated(s["k"], pos, *turn).to(dt)
    s["vc"].view(-1, c["hkv"], c["d"])[slots] = s["v"]
    return q, s["kc"], s["vc"]


def _gathered(s, cache, length):
    """Every row's context side by side, in 32 bits: [rows, Hkv, length, D] (what lies past a context is masked)."""
    x = cache[s["tables"].clamp(min=0).to(torch.int64)].flatten(1, 2)[:, :length]
    return x.float().transpose(1, 2)


def _weighted(s, scores, visible, distance, values):
    """softmax of the capped and biased scores [..., Hkv, G, Q, K] over the visible keys, times the values."""
    c = s["case"]
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    if s["slopes"] is not None:
        scores = scores - s["slopes"].view(c["hkv"], -1, 1, 1) * distance
    scores = scores.masked_fill(~visible, float("-inf"))
    weights = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    total = weights.sum(dim=-1, keepdim=True)
    return torch.matmul(weights.flatten(2, 3), values) / total.flatten(2, 3)


def _plain_decode(s):
    c = s["case"]
    n, hkv, d = c["seqs"], c["hkv"], c["d"]
    q = s["q"].float().view(n, hkv, -1, d)
    scores = torch.matmul(q, _gathered(s, s["kc"], s["max_ctx"]).transpose(2, 3)) * s["scale"]
    j = torch.arange(s["max_ctx"], device=DEV)
    back = s["ctx"].to(torch.int64)[:, None] - 1 - j            # how far a key lies behind the new token
    visible = back >= 0
    if c["window"]:
        visible = visible & (back < c["window"])
    out = _weighted(s, scores.unsqueeze(3), visible.view(n, 1, 1, 1, -1), back.abs().float().view(n, 1, 1, 1, -1),
                    _gathered(s, s["vc"], s["max_ctx"]))
    return out.reshape(n, -1, d).to(s["q"].dtype)


def _plain_prefill(s):
    c = s["case"]
    n, hkv, hq, d, mq, mk = c["seqs"], c["hkv"], c["hq"], c["d"], s["max_q"], s["max_k"]
    seq, pos = _rows_of(s["cu_q"], s["cu_k"], s["q"].shape[0])
    local = torch.arange(s["q"].shape[0], device=DEV) - s["cu_q"][seq]
    q = torch.zeros(n, mq, hq, d, device=DEV)
    q[seq, local] = s["q"].float()
    q = q.view(n, mq, hkv, -1, d).permute(0, 2, 3, 1, 4)        # [n, Hkv, G, Q, D]
    scores = torch.matmul(q.flatten(2, 3), _gathered(s, s["kc"], mk).transpose(2, 3)) * s["scale"]
    place = torch.zeros(n, mq, dtype=torch.int64, device=DEV)
    place[seq, local] = pos
    j = torch.arange(mk, device=DEV)
    back = place[:, :, None] - j
    visible = back >= 0
    if c["window"]:
        visible = visible & (back < c["window"])
    if s["prefix"] is not None:
        visible = visible | (j < s["prefix"].to(torch.int64)[:, None, None])
    out = _weighted(s, scores.view(n, hkv, -1, mq, mk), visible.view(n, 1, 1, mq, mk),
                    back.abs().float().view(n, 1, 1, mq, mk), _gathered(s, s["vc"], mk))
    out = out.view(n, hkv, -1, mq, d).permute(0, 3, 1, 2, 4).reshape(n, mq, hq, d)
    return out[seq, local].to(s["q"].dtype)


EOS = 2


def _plain_beam(s):
    """The `keep` best continuations of every request; values next to one another are told apart in 64 bits."""
    c = s["case"]
    n, b, v = c["reqs"], c["beams"], c["vocab"]
    x = s["logits"].to(torch.float64)
    top = x.amax(dim=1, keepdim=True)
    norm = top + torch.log(torch.exp(x - top).sum(dim=1, keepdim=True))
    total = (s["scores"].to(torch.float64).view(-1, 1) - norm + x).view(n, b, v)
    if s["finished"] is not None:          # an ended beam stays as it is: its end id again, at no cost
        ended = torch.full((n, b, v), float("-inf"), dtype=torch.float64, device=x.device)
        ended[:, :, EOS] = s["scores"].to(torch.float64)
        total = torch.where(s["finished"].bool()[:, :, None], ended, total)
    best, at = torch.sort(total.view(n, b * v), dim=1, descending=True, stable=True)
    best, at = best[:, :c["keep"]], at[:, :c["keep"]]
    none = best == float("-inf")           # fewer continuations than asked for: no beam and no id in their place
    at = torch.where(none, -1, at)
    return best.float(), (at // v).to(torch.int32), torch.where(none, -1, at % v).to(torch.int32)


# --------------------------------------------------------------------- run
def _own(s):
    import paged_kv_decode_store_gb300 as pk
    c = s["case"]
    kind = c["kind"]
    if kind == "rope":
        return pk.rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                       mscale=s["mscale"])
    if kind == "rope_decode":
        q = pk.rope_store_paged(s["q"], s["k"], s["v"], s["tables"], s["ctx"], s["inv_freq"], s["kc"], s["vc"],
                                interleaved=c["interleaved"], mscale=s["mscale"])
        return q, s["kc"], s["vc"]
    if kind == "rope_prefill":
        q = pk.rope_store_prefill(s["q"], s["k"], s["v"], s["tables"], s["cu_q"], s["cu_k"], s["inv_freq"], s["kc"],
                                  s["vc"], interleaved=c["interleaved"], mscale=s["mscale"])
        return q, s["kc"], s["vc"]
    if kind == "decode":
        return pk.paged_decode_attention(s["q"], s["kc"], s["vc"], s["tables"], s["ctx"], s["max_ctx"], s["scale"],
                                         workspace=s["workspace"], window=c["window"], softcap=c["softcap"],
                                         alibi_slopes=s["slopes"])
    if kind == "prefill":
        return pk.prefill_attention(s["q"], s["kc"], s["vc"], s["tables"], s["cu_q"], s["cu_k"], s["max_q"],
                                    s["scale"], window=c["window"], softcap=c["softcap"], alibi_slopes=s["slopes"],
                                    prefix_lens=s["prefix"])
    return pk.beam_search_step(s["logits"], s["scores"], c["keep"], finished=s["finished"], eos_id=EOS)


def run(s):
    if own:
        return _own(s)
    kind = s["case"]["kind"]
    if kind == "decode":
        return _plain_decode(s)
    if kind == "prefill":
        return _plain_prefill(s)
    if kind == "beam":
        return _plain_beam(s)
    return _plain_rope(s)


# -------------------------------------------------------------------- work
def work(case):
    e = SIZE[case["dtype"]]
    kind = case["kind"]
    if kind == "beam":
        rows = case["reqs"] * case["beams"]
        n = rows * case["vocab"]
        return {"bytes": n * e + rows * 5 + case["reqs"] * case["keep"] * 12, "flops": 4 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if kind.startswith("rope"):
        if kind == "rope":
            t = case["tokens"]
            return {"bytes": t * (2 * (hq + hkv) * d * e + 8), "flops": t * (hq + hkv) * case["rot"] * 3}
        t = case["seqs"] if kind == "rope_decode" else sum(_query_lengths(case))
        return {"bytes": t * (2 * (hq + 2 * hkv) * d * e + 8), "flops": t * (hq + hkv) * case["rot"] * 3}
    if kind == "decode":
        lens = _lengths(case, case["lo"], case["hi"], case["seqs"], "ctx")
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        return {"bytes": 2 * seen * hkv * d * e + 2 * len(lens) * hq * d * e + 4 * sum(-(-n // case["bs"]) for n in lens),
                "flops": 4 * seen * hq * d}
    qlens, cached = _query_lengths(case), _cached_lengths(case)
    lens = [q + c for q, c in zip(qlens, cached)]
    prefix = _prefix_lengths(case, lens) if case["prefix"] else [0] * len(lens)
    pairs = 0
    for q, c, f in zip(qlens, cached, prefix):
        for p in range(c, c + q):
            first = max(0, p + 1 - case["window"]) if case["window"] else 0
            pairs += p + 1 - first if f == 0 else f + max(0, p + 1 - max(first, f))
    read = [k if f or not case["window"] else min(k, q + case["window"] - 1) for q, k, f in zip(qlens, lens, prefix)]
    return {"bytes": 2 * sum(read) * hkv * d * e + 2 * sum(qlens) * hq * d * e, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- exact
def _turn64(x, pos, inv, interleaved, mscale):
    """Each pair as a complex number, times mscale e^(i position inv_freq)."""
    y = x.to(torch.float64).clone()
    m = inv.shape[0]
    one = slice(0, 2 * m, 2) if interleaved else slice(0, m)
    two = slice(1, 2 * m, 2) if interleaved else slice(m, 2 * m)
    z = torch.complex(y[..., one], y[..., two])
    phase = pos.to(torch.float64)[:, None] * inv[None]
    z = z * torch.polar(torch.full_like(phase, mscale), phase)[:, None, :]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["case"]
    args = (s["inv_freq"], c["interleaved"], s["mscale"])
    if c["kind"] == "rope":
        return _turn64(s["q"], s["positions"], *args), _turn64(s["k"], s["positions"], *args)
    if c["kind"] == "rope_decode":
        rows = [(i, n - 1) for i, n in enumerate(s["ctx"].tolist())]
    else:
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        rows = []
        for i in range(c["seqs"]):
            end, new = ck[i + 1] - ck[i], cq[i + 1] - cq[i]
            rows += [(i, p) for p in range(end - new, end)]
    tables = s["tables"].tolist()
    pos = torch.tensor([p for _, p in rows], device=DEV)
    block = torch.tensor([tables[i][p // c["bs"]] for i, p in rows], device=DEV)
    kc, vc = s["kc"].double(), s["vc"].double()
    kc[block, pos % c["bs"]] = _turn64(s["k"], pos, *args)
    vc[block, pos % c["bs"]] = s["v"].double()
    return _turn64(s["q"], pos, *args), kc, vc


def _exact_attention(s):
    """One sequence, and one KV head of it, at a time."""
    c = s["case"]
    hkv, d, group = c["hkv"], c["d"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if c["kind"] == "decode":
        spans = [(i, i + 1, n) for i, n in enumerate(s["ctx"].tolist())]
        prefix = [0] * len(spans)
    else:
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        spans = [(cq[i], cq[i + 1], ck[i + 1] - ck[i]) for i in range(c["seqs"])]
        prefix = s["prefix"].tolist() if s["prefix"] is not None else [0] * len(spans)
    for i, (a, b, n) in enumerate(spans):
        ids = s["tables"][i, :-(-n // c["bs"])].to(torch.int64)
        key, val = (x[ids].reshape(-1, hkv, d)[:n].double() for x in (s["kc"], s["vc"]))
        p = torch.arange(n - (b - a), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        seen = j <= p
        if c["window"]:
            seen = seen & (j > p - c["window"])
        seen = seen | (j < prefix[i])
        for h in range(hkv):
            q = s["q"][a:b, h * group:(h + 1) * group].double()             # [rows, group, d]
            x = torch.einsum("rgd,nd->grn", q, key[:, h]) * s["scale"]
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if s["slopes"] is not None:
                x = x - s["slopes"][h * group:(h + 1) * group].double()[:, None, None] * (p - j).abs()
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            out[a:b, h * group:(h + 1) * group] = torch.einsum("grn,nd->rgd", torch.softmax(x, dim=-1), val[:, h])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("rope"):
        return _exact_rope(s)
    if case["kind"] != "beam":
        return _exact_attention(s)
    scores = []
    for r in range(case["reqs"]):
        found = []
        for b in range(case["beams"]):
            before = s["scores"][r, b].double()
            if s["finished"] is not None and bool(s["finished"][r, b]):
                found.append(before.view(1))
                continue
            x = torch.log_softmax(s["logits"][r * case["beams"] + b].double(), dim=0)
            found.append(before + torch.topk(x, min(case["keep"], x.shape[0])).values)
        found.append(torch.full((case["keep"],), -math.inf, dtype=torch.float64, device=DEV))   # where there are fewer
        scores.append(torch.topk(torch.cat(found), case["keep"]).values)
    return torch.stack(scores), None, None
