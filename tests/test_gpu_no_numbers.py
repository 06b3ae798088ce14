"""A NaN in a query, or in a key that a row sees, makes that row NaN however its keys are cut over the card; in decode
every weight that it counts too.  Other rows keep every bit."""
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_score_mod import DT, EPS, cache_of
from test_gpu_tree import cumulative, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"

# few rows a tree, many, fp32 arithmetic in 16 bits and fp32
TREES = [("bf16", 3, 1, 128, 3, 4), ("f16", 2, 1, 64, 3, 9), ("bf16", 20, 1, 64, 3, 5), ("f16", 24, 1, 128, 3, 12),
         ("bf16", 2, 1, 64, 1, 4), ("f32", 4, 1, 64, 1, 10)]


@pytest.mark.parametrize("cached", [100, 20000])
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(map(str, c)))
def test_trees(case, cached):
    """Over 20,000 keys a CTA has a tile or two, and the merge joins what they leave."""
    pk = require_gpu()
    name, hq, hkv, d, path, n = case
    dt = DT[name]
    kc, vc, tables, _ = cache_of([cached + n, 50 + n], hkv, d, 16, dt, 1)
    q = torch.randn(2 * n, hq, d, generator=torch.Generator().manual_seed(2)).to(dt).to(DEV)
    star = ints(([-1] + [0] * (n - 1)) * 2)
    call = lambda q, kc: pk.tree_attention(q, kc, vc, tables, cumulative([n, n]), cumulative([cached + n, 50 + n]), star, n,
                                           d ** -0.5, path=path)
    plain = call(q, kc)
    assert torch.isfinite(plain).all()
    bad = q.clone()
    bad[2, 1, 5] = float("nan")
    got = call(bad, kc)
    assert got[2, 1].isnan().all()
    got[2, 1] = plain[2, 1]
    assert torch.equal(got, plain)
    for key in (0, cached // 2 + 3, cached - 1):             # every row of the first tree sees it
        k2 = kc.clone()
        k2[tables[0, key // 16], key % 16, 0, 7] = float("nan")
        got = call(q, k2)
        assert got[:n].isnan().all(), key
        assert torch.equal(got[n:], plain[n:])
    k2 = kc.clone()                                          # a leaf's own row: nobody else's
    k2[tables[0, (cached + n - 1) // 16], (cached + n - 1) % 16, 0, 7] = float("nan")
    got = call(q, k2)
    assert got[n - 1].isnan().all()
    got[n - 1] = plain[n - 1]
    assert torch.equal(got, plain)

DECODE = [("bf16", 16, 8, 128, 0), ("f16", 16, 8, 64, 1), ("f32", 4, 2, 64, 0), ("bf16", 6, 1, 128, 0)]


@pytest.mark.parametrize("ctx", [16, 1601, 20001])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c)))
def test_decode_with_weights(case, ctx):
    """1,601 keys of one row: a chunk of 16 for each CTA, and one key in the last."""
    pk = require_gpu()
    name, hq, hkv, d, path = case
    dt, G = DT[name], hq // hkv
    kc, vc, tables, _ = cache_of([ctx], hkv, d, 16, dt, 3)
    q = torch.randn(1, hq, d, generator=torch.Generator().manual_seed(4)).to(dt).to(DEV)

    def call(q, kc):
        w = torch.zeros(1, hkv, ctx, device=DEV)
        out, _ = pk.paged_decode_attention_weights(q, kc, vc, tables, ints([ctx]), ctx, d ** -0.5, w, path=path)
        return out, w

    plain = call(q, kc)
    assert all(torch.isfinite(x).all() for x in plain)

    def others_as_before(got, hk):
        for x, y, heads in ((got[0], plain[0], slice(hk * G, hk * G + G)), (got[1], plain[1], slice(hk, hk + 1))):
            x = x.clone()
            x[:, heads] = y[:, heads]
            assert torch.equal(x, y)

    bad = q.clone()
    bad[0, 0, 9] = float("nan")
    got = call(bad, kc)
    assert got[0][0, 0].isnan().all() and got[1][0, 0].isnan().all()
    others_as_before(got, 0)
    for key in (0, ctx // 2, ctx - 1):
        k2, hk = kc.clone(), hkv - 1
        k2[tables[0, key // 16], key % 16, hk, 3] = float("nan")
        got = call(q, k2)
        assert got[0][0, hk * G:].isnan().all() and got[1][0, hk].isnan().all(), key
        others_as_before(got, hk)


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c)))
def test_keys_at_minus_infinity(case):
    """Scores of -inf, whole pieces of a row among them: those keys weigh nothing, the others what they do without them."""
    pk = require_gpu()
    name, hq, hkv, d, path = case
    dt, G, ctx = DT[name], hq // hkv, 1601
    kc, vc, tables, _ = cache_of([ctx], hkv, d, 16, dt, 5)
    q = torch.randn(1, hq, d, generator=torch.Generator().manual_seed(6)).to(dt).to(DEV)
    q[:, :, 11] = q[:, :, 11].abs() + 1
    rows = [(int(tables[0, j // 16]), j % 16) for j in range(ctx)]
    gone = [j for j in range(ctx) if j < 40 or 800 <= j < 950 or j == ctx - 1]
    stay = [j for j in range(ctx) if j not in set(gone)]
    for j in gone:
        kc[rows[j][0], rows[j][1], :, 11] = float("-inf")
    w = torch.zeros(1, hkv, ctx, device=DEV)
    out, _ = pk.paged_decode_attention_weights(q, kc, vc, tables, ints([ctx]), ctx, d ** -0.5, w, path=path)
    assert torch.all(w[:, :, gone] == 0)
    k, v = (torch.stack([x[b, r] for b, r in (rows[j] for j in stay)]).double().cpu().numpy() for x in (kc, vc))
    u_p = 0.0 if name == "f32" or path == 1 or hkv not in (8, 16) else EPS[dt] / 2
    for h in range(hq):
        qh = q[0, h].double().cpu().numpy()
        # (position: without a bias only which keys there are counts)
        want, bound = oracle.scores.attend(qh, k[:, h // G], v[:, h // G], len(stay) - 1, d ** -0.5, u_p=u_p, eps=EPS[dt],
                                           tiny=2.0 ** -24 if name == "f16" else 0.0)
        assert (abs(out[0, h].double().cpu().numpy() - want) <= bound).all(), h
    for r in range(hkv):
        total, bound = 0.0, 0.0
        for h in range(r * G, r * G + G):
            x, b = oracle.drafts.given(q[0, h].double().cpu().numpy(), k[:, r], len(stay), d ** -0.5)
            total, bound = total + x, bound + b
        off = abs(w[0, r, stay].double().cpu().numpy() - total)
        assert (off <= bound + (G + 1) * 2.0 ** -24 * total).all(), r
