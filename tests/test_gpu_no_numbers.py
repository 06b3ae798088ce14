"""A NaN in a query, or in a key that a row sees, makes that row NaN however its keys are cut over the card.  Other rows
keep every bit."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_score_mod import DT, cache_of
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
