"""Seeded random shapes of the modified attention (decode and prefill) and of
beam search against the float64 oracles: head counts and groups, types, block
sizes, lengths from nothing to hundreds, caps, slopes, windows and prefixes."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_beam import check as check_beams
from test_gpu_score_mod import DEV, DT, cache_of, slopes_for, tolerances

pytestmark = pytest.mark.gpu


def modifiers(rng):
    cap = float(rng.choice([0.0, 0.0, 1.5, 7.0, 50.0]))
    kind = rng.choice([None, "geometric", "mixed"])
    if cap == 0.0 and kind is None:
        kind = "geometric"
    return cap, kind, int(rng.choice([0, 0, 1, 40, 200]))


def heads(rng, dt):
    if dt == "f32":
        return int(rng.choice([1, 2, 4, 5])), int(rng.choice([1, 2, 3, 4])), 64
    return int(rng.choice([1, 2, 4, 8, 16])), int(rng.choice([1, 2, 3, 5, 6, 8])), int(rng.choice([64, 128]))


@pytest.mark.parametrize("seed", range(20))
def test_decode(seed):
    pk = require_gpu()
    rng = np.random.default_rng(seed)
    name = str(rng.choice(["f32", "f16", "bf16"]))
    hkv, group, d = heads(rng, name)
    if hkv == 16:
        d = 64
    dt, hq, bs = DT[name], hkv * group, int(rng.choice([16, 32, 64, 256]))
    ctx = [int(x) for x in rng.choice([0, 1, 2, 15, 16, 17, 63, 130, 257, 600], size=int(rng.integers(1, 9)))]
    cap, kind, window = modifiers(rng)
    kc, vc, tables, rows = cache_of(ctx, hkv, d, bs, dt, seed)
    q = (2 * torch.randn(len(ctx), hq, d, generator=torch.Generator().manual_seed(seed))).to(dt)
    dev_slopes, slopes = slopes_for(hq, kind)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pk.paged_decode_attention(q.to(DEV), kc, vc, tables, torch.tensor(ctx, dtype=torch.int32, device=DEV),
                                    max(max(ctx), 1), d ** -0.5, window=window, softcap=cap, alibi_slopes=dev_slopes,
                                    err=err)
    assert err.item() == 0
    got, tol = out.double().cpu().numpy(), tolerances(dt, name != "f32" and hkv in (8, 16))
    for i, n in enumerate(ctx):
        for h in range(hq):
            k, v = (x[:, h // group] for x in rows[i])
            want, bound = oracle.scores.attend(q[i, h].double().numpy(), k, v, n - 1, d ** -0.5, cap, slopes[h], window,
                                               **tol)
            assert np.all(np.abs(got[i, h] - want) <= bound), (i, h)


@pytest.mark.parametrize("seed", range(24))
def test_prefill(seed):
    pk = require_gpu()
    rng = np.random.default_rng(100 + seed)
    name = str(rng.choice(["f16", "bf16", "f16", "bf16", "f32"]))
    hkv, group, d = heads(rng, name)
    dt, hq, bs = DT[name], hkv * group, int(rng.choice([8, 16, 64, 128, 256]))
    n = int(rng.integers(1, 7))
    qlen = [int(x) for x in rng.choice([0, 1, 3, 21, 64, 100, 190], size=n)]
    klen = [a + int(b) for a, b in zip(qlen, rng.choice([0, 0, 1, 77, 128, 350], size=n))]
    if not sum(qlen):
        qlen[0], klen[0] = 5, klen[0] + 5
    cap, kind, window = modifiers(rng)
    prefix = [int(rng.integers(-3, k + 30)) for k in klen] if rng.random() < 0.5 else None
    kc, vc, tables, rows = cache_of(klen, hkv, d, bs, dt, seed)
    q = (2 * torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(seed))).to(dt)
    cq, ck = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (qlen, klen))
    dev_slopes, slopes = slopes_for(hq, kind)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pl = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    out = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, max(qlen), d ** -0.5, window=window, err=err,
                               softcap=cap, alibi_slopes=dev_slopes, prefix_lens=pl)
    assert err.item() == 0
    got, tol, t0 = out.double().cpu().numpy(), tolerances(dt, name != "f32"), 0
    for i, k_all in enumerate(klen):
        open_to = 0 if prefix is None else min(max(prefix[i], 0), k_all)
        for j in {0, qlen[i] - 1, *range(seed % 7, qlen[i], 13)} if qlen[i] else ():
            for h in {(j * 5) % hq, hq - 1, 0}:
                k, v = (x[:, h // group] for x in rows[i])
                want, bound = oracle.scores.attend(q[t0 + j, h].double().numpy(), k, v, k_all - qlen[i] + j, d ** -0.5, cap,
                                                   slopes[h], window, open_to, **tol)
                assert np.all(np.abs(got[t0 + j, h] - want) <= bound), (i, j, h)
        t0 += qlen[i]


@pytest.mark.parametrize("seed", range(16))
def test_beams(seed):
    pk = require_gpu()
    rng = np.random.default_rng(200 + seed)
    dt = DT[str(rng.choice(["f32", "f16", "bf16"]))]
    n, b, keep = int(rng.integers(1, 6)), int(rng.choice([1, 2, 3, 4, 7, 16])), int(rng.choice([1, 2, 5, 16, 64]))
    V = int(rng.choice([1, 2, 65, 511, 513, 4096, 20000, 70001]))
    g = torch.Generator().manual_seed(seed)
    wide = torch.full((n * b, V + int(rng.integers(0, 9))), float("nan"), dtype=dt, device=DEV)      # strided rows
    wide[:, :V] = (float(rng.choice([0.5, 3.0, 20.0])) * torch.randn(n * b, V, generator=g)).to(dt).to(DEV)
    logits = wide[:, :V]
    if rng.random() < 0.5:
        logits[torch.rand(n * b, V, generator=g).to(DEV) < 0.6] = float("-inf")
    scores = (-9 * torch.rand(n, b, generator=g)).to(DEV)
    finished, eos = None, -1
    if rng.random() < 0.5:
        finished, eos = (torch.rand(n, b, generator=g) < 0.3).to(torch.uint8).to(DEV), int(rng.integers(0, V))
    check_beams(pk.beam_search_step(logits, scores, keep, finished=finished, eos_id=eos), logits, scores, keep, finished, eos)
