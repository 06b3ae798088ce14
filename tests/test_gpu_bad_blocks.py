"""Block ids of every wrong kind read as zeros and are reported, whatever bits they have: the smallest int32 too,
in tiles that every row sees, where a stage holds an earlier tile's rows."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_score_mod import cache_of
from test_gpu_tree import cumulative, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"
IDS = [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 31 - 1]


def with_zero_block(dt, hkv, d, klen, seed):
    """Caches, tables and the id of a block of zeros that no table has."""
    kc, vc, tables, _ = cache_of(klen, hkv, d, 16, dt, seed)
    zero = next(b for b in range(kc.shape[0]) if not (tables == b).any())
    kc[zero], vc[zero] = 0, 0
    return kc, vc, tables, zero


def same_with_every_bad_id(pk, call, tables, at, zero):
    """call(tables, err) with each wrong id in the same places gives what a block of zeros gives there, and says so."""
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = tables.clone()
    for i, j in at:
        t[i, j] = zero
    want = call(t, err)
    assert err.item() == 0 and torch.isfinite(want).all()
    for bad in IDS:
        for i, j in at:
            t[i, j] = bad
        err.zero_()
        got = call(t, err)
        assert err.item() == pk.ERR_BLOCK_ID, bad
        assert torch.equal(got, want), bad


@pytest.mark.parametrize("case", [("bf16", 16, 2, 128, 3, 4), ("f16", 4, 2, 64, 3, 4), ("bf16", 64, 2, 128, 3, 9), ("f16", 40, 1, 64, 3, 20),
                                  ("f32", 4, 2, 64, 1, 4)], ids=lambda c: "-".join(map(str, c)))
def test_trees(case):
    pk = require_gpu()
    name, hq, hkv, d, path, n = case
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]
    klen = [3000, 777]
    kc, vc, tables, zero = with_zero_block(dt, hkv, d, klen, 3)
    q = torch.randn(2 * n, hq, d, generator=torch.Generator().manual_seed(5)).to(dt).to(DEV)
    parents = ints([-1] + list(range(n - 1)) + [-1] + [0] * (n - 1))
    call = lambda t, err: pk.tree_attention(q, kc, vc, t, cumulative([n, n]), cumulative(klen), parents, n, d ** -0.5, err=err,
                                            path=path)
    same_with_every_bad_id(pk, call, tables, [(0, 0), (0, 100), (0, 101), (0, 150), (1, 30)], zero)


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("case", [("bf16", 16, 2, 128), ("f16", 4, 2, 64)], ids=lambda c: "-".join(map(str, c)))
def test_prefill(case, softcap):
    pk = require_gpu()
    name, hq, hkv, d = case
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[name]
    qlen, klen = [40, 200], [3000, 777]
    kc, vc, tables, zero = with_zero_block(dt, hkv, d, klen, 4)
    q = torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(6)).to(dt).to(DEV)
    call = lambda t, err: pk.prefill_attention(q, kc, vc, t, cumulative(qlen), cumulative(klen), max(qlen), d ** -0.5, err=err,
                                               path=pk.PATH_TC, softcap=softcap)
    same_with_every_bad_id(pk, call, tables, [(0, 0), (0, 100), (0, 101), (0, 150), (1, 30)], zero)


@pytest.mark.parametrize("klen", [-2 ** 31, -2 ** 31 + 3, -1, 0, 2, 2 ** 31 - 1])
@pytest.mark.parametrize("case", [("bf16", 16, 3), ("bf16", 64, 3), ("f32", 4, 1)], ids=lambda c: "-".join(map(str, c)))
def test_lengths_that_no_tree_has(case, klen):
    """A k_len below the drafts' number or past the table, whatever its difference wraps to, leaves its sequence out."""
    pk = require_gpu()
    name, hq, path = case
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[name]
    kc, vc, tables, _ = cache_of([100, 60], 2, 64, 16, dt, 8)
    n = 20 if hq == 64 else 3
    q = torch.randn(2 * n, hq, 64, generator=torch.Generator().manual_seed(9)).to(dt).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    chain = ints((list(range(-1, n - 1))) * 2)
    cu_k = torch.tensor([-60, 0, klen], dtype=torch.int64).to(torch.int32).to(DEV)       # the first sequence is a good one
    cu_q = cumulative([n, n])
    out = torch.full_like(q, 7.0)
    pk.tree_attention(q, kc, vc, tables, cu_q, cu_k, chain, n, 0.125, out=out, err=err, path=path)
    assert err.item() == pk.ERR_CONTEXT
    assert torch.all(out[n:] == 7.0) and torch.isfinite(out[:n]).all() and not torch.all(out[:n] == 7.0)
    if klen != 2 ** 31 - 1:                                  # (the walk has no table: any length from n on is one)
        err.zero_()
        ids = torch.zeros(2 * n, dtype=torch.int32, device=DEV)
        _, first, counts, _ = pk.tree_accept(ids, chain, ids, cu_q, cu_k, 4, err=err)
        assert err.item() == pk.ERR_CONTEXT and counts.tolist() == [min(n, 4), 0] and first.tolist() == [60 - n, 0]
