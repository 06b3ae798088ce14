"""Rotary store, attention with modified scores, beam selection and the block
tables that follow it, run together as a beam search decodes: prompts that
share a cached prefix, then steps in which beams are kept, cloned and dropped
and partial blocks copied before they are written.

The rows a beam finds through its block table are its own tokens' keys and
values, turned by their positions (within fp32 and one rounding of the cache's
type); its attention is that of the float64 oracle over them; the beams chosen
are the oracle's on the same logits."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_beam import check as check_beams

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.double().cpu().numpy()


CASES = [("bf16", 8, 2, 64, 16, dict(softcap=3.0), False), ("f16", 12, 2, 128, 16, dict(alibi=True), False),
         ("f32", 8, 2, 64, 16, dict(softcap=4.0, alibi=True), True), ("bf16", 4, 4, 128, 16, dict(softcap=2.0), True)]


@pytest.mark.parametrize("dtype,hq,hkv,D,bs,mod,interleaved", CASES, ids=[f"{c[0]}-{c[1]}x{c[3]}" for c in CASES])
def test_beam_search(dtype, hq, hkv, D, bs, mod, interleaved):
    pk = require_gpu()
    dt, dev, V, B, steps = DT[dtype], "cuda", 61, 3, 21
    fi = torch.finfo(dt)
    g = torch.Generator().manual_seed(hq * D)
    table_qkv = (1.2 * torch.randn(V, hq + 2 * hkv, D, generator=g)).to(dt).to(dev)   # a token's projected rows
    head = torch.randn(hq * D, V, generator=g).to(dev) / (hq * D) ** 0.5 * 3
    scale, cap = D ** -0.5, mod.get("softcap", 0.0)
    slopes = (2.0 ** -torch.arange(1, hq + 1, dtype=torch.float32)).to(dev) if mod.get("alibi") else None
    inv, mscale = pk.rope_inv_freq(D, device=dev)
    args = dict(softcap=cap, alibi_slopes=slopes)
    kc = torch.full((64, bs, hkv, D), float("nan"), dtype=dt, device=dev)
    vc = torch.full_like(kc, float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    bm = pk.BlockManager(64, bs)
    common = torch.randint(0, V, (bs + 3,), generator=g).tolist()
    prompts = [common + torch.randint(0, V, (n,), generator=g).tolist() for n in (7, 18)]

    def padded(tables):
        t = torch.full((len(tables), max(map(len, tables))), -1, dtype=torch.int32)
        for i, row in enumerate(tables):
            t[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        return t.to(dev)

    def cached_rows(history, table):
        """A sequence's keys and values through its table, checked against its tokens'."""
        n = len(history)
        at = torch.tensor([table[p // bs] * bs + p % bs for p in range(n)], device=dev)
        k, v = f64(kc.view(-1, hkv, D)[at]), f64(vc.view(-1, hkv, D)[at])
        rows = table_qkv[torch.tensor(history, device=dev)]
        assert np.array_equal(v, f64(rows[:, hq + hkv:]))
        raw = f64(rows[:, hq:hq + hkv])
        want = oracle.rotary.rotate(raw, range(n), f64(inv), interleaved, mscale)
        bound = oracle.rotary.error_bound(raw, want, D, interleaved, mscale, fi.eps, fi.tiny)
        assert (np.abs(k - want) <= bound).all()
        return k, v

    def check_attention(q, out, history, table):
        k, v = cached_rows(history, table)
        p = len(history) - 1
        u_p = 0.0 if dtype == "f32" else fi.eps / 2
        for h in range(hq):
            slope = 0.0 if slopes is None else float(slopes[h])
            want, bound = oracle.scores.attend(f64(q)[h], k[:, h * hkv // hq], v[:, h * hkv // hq], p, scale, cap, slope,
                                               u_p=u_p, eps=fi.eps, tiny=fi.tiny)
            assert (np.abs(f64(out)[h] - want) <= bound).all(), (h, np.abs(f64(out)[h] - want).max())

    # prompts: the second one finds the first block in the cache
    tables, new, lens = [], [], []
    for prompt in prompts:
        table, cached = bm.allocate(prompt)
        tables.append(table)
        new.append(prompt[cached:])
        lens.append(len(prompt))
    assert len(new[1]) == lens[1] - bs
    rows = table_qkv[torch.tensor(sum(new, []), device=dev)]
    cu_q = torch.tensor(np.cumsum([0] + [len(x) for x in new]), dtype=torch.int32, device=dev)
    cu_k = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=dev)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    q = pk.rope_store_prefill(q, k, v, padded(tables), cu_q, cu_k, inv, kc, vc, interleaved, mscale, err=err)
    out = pk.prefill_attention(q, kc, vc, padded(tables), cu_q, cu_k, max(map(len, new)), scale, err=err, **args)
    last = (cu_q[1:] - 1).long()
    for i, prompt in enumerate(prompts):
        check_attention(q[last[i]], out[last[i]], prompt, tables[i])

    # beams: clones of their prompt, the first one alive
    n = len(prompts)
    history = [list(p) for p in prompts for _ in range(B)]
    tables = [t if b == 0 else bm.fork(t) for t in tables for b in range(B)]
    scores = torch.full((n, B), float("-inf"), device=dev)
    scores[:, 0] = 0.0
    logits = (out[last].float().reshape(n, -1) @ head).repeat_interleave(B, 0)
    cloned = copied = 0
    for _ in range(steps):
        got = pk.beam_search_step(logits, scores, B)
        check_beams(got, logits, scores, B)
        scores, parents, tokens = got
        parents = (parents.cpu() + B * torch.arange(n).view(n, 1)).flatten().tolist()
        cloned += len(parents) - len(set(parents))
        tables = bm.reorder(tables, parents)
        history = [history[p] + [t] for p, t in zip(parents, tokens.cpu().flatten().tolist())]
        copies = []
        for i, row in enumerate(history):
            tables[i], copy = bm.append(row, tables[i])
            assert tables[i] is not None
            if copy:
                copies.append(copy)
        if copies:
            copied += len(copies)
            src, dst, cnt = (torch.tensor(x, dtype=torch.int32, device=dev) for x in zip(*copies))
            pk.copy_blocks(kc, vc, src, dst, cnt, err=err)
        rows = table_qkv[tokens.flatten().long()]
        ctx = torch.tensor([len(x) for x in history], dtype=torch.int32, device=dev)
        bt = padded(tables)
        q = pk.rope_store_paged(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], bt, ctx, inv, kc, vc, interleaved,
                                mscale, err=err)
        out = pk.paged_decode_attention(q, kc, vc, bt, ctx, max(map(len, history)), scale, err=err, **args)
        for i, row in enumerate(history):
            check_attention(q[i], out[i], row, tables[i])
        logits = out.float().reshape(n * B, -1) @ head
    assert int(err.item()) == 0
    assert cloned > 0 and copied > 0                       # beams split and shared partial blocks
    for t in tables:
        bm.release(t)
    assert bm.num_free() == 64
