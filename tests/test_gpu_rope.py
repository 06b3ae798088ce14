"""Rotary positions on the GPU against the float64 oracle: every layout, part
of the head, type and stride; far positions; the fused stores' cache bits."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# machine epsilon and smallest subnormal of each type
ROUND = {torch.float32: (2.0 ** -23, 0.0), torch.float16: (2.0 ** -10, 2.0 ** -24), torch.bfloat16: (2.0 ** -7, 0.0)}


def close(got, x, positions, inv, interleaved, mscale):
    """got [T, H, D] is x rotated, within the bound that the oracle derives."""
    x = x.double().cpu().numpy()
    y = oracle.rotary.rotate(x, positions, inv, interleaved, mscale)
    eps, tiny = ROUND[got.dtype]
    bound = oracle.rotary.error_bound(x, y, 2 * len(inv), interleaved, mscale, eps, tiny)
    off = np.abs(got.double().cpu().numpy() - y)
    assert np.all(off <= bound), (float((off - bound).max()), np.argwhere(off > bound)[:4])


def projected(T, hq, hkv, d, dt, seed, pad=0):
    """q, k, v as slices of one projected tensor (rows `pad` heads longer than they need)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hq + 2 * hkv + pad, d, generator=g).to(dt).to(DEV)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


SHAPES = [  # T, hq, hkv, d, rot
    (1, 1, 1, 64, 64), (3, 4, 2, 64, 32), (5, 16, 16, 64, 48), (2, 48, 8, 128, 128), (7, 3, 1, 128, 112),
    (4, 8, 2, 64, 2), (3, 2, 1, 128, 18), (2, 5, 5, 256, 64), (2, 1, 1, 512, 512), (3, 40, 3, 32, 20), (1, 7, 0, 64, 64),
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_rope_matches_the_oracle(shape, dt, interleaved):
    pk = require_gpu()
    T, hq, hkv, d, rot = shape
    q, k, _ = projected(T, hq, hkv, d, DT[dt], 1, pad=hkv % 2)
    inv, m = pk.rope_inv_freq(rot)
    pos = [0, 1, 131071, 2 ** 22 + 7, -5, 2 ** 40 + 3, 999][:T]
    keep = q.clone(), k.clone()
    qo, ko = pk.rope(q, k if hkv else None, torch.tensor(pos, device=DEV), inv, interleaved=interleaved)
    close(qo, q, pos, inv.tolist(), interleaved, m)
    if hkv:
        close(ko, k, pos, inv.tolist(), interleaved, m)
    else:
        assert ko is None
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])


@pytest.mark.parametrize("scaling", ["linear", "ntk", "parts"])
def test_rope_scaled_for_long_contexts(scaling):
    pk = require_gpu()
    q, k, _ = projected(6, 4, 2, 64, torch.float32, 2)
    inv, m = pk.rope_inv_freq(64, 500000.0, scaling, 16.0, 8192)
    pos = [0, 8191, 8192, 100000, 131071, 2 ** 31 + 5]
    qo, ko = pk.rope(q, k, torch.tensor(pos, device=DEV), inv, mscale=m)
    close(qo, q, pos, inv.tolist(), False, m)
    close(ko, k, pos, inv.tolist(), False, m)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [64, 48, 18])
def test_rope_in_place_is_the_same_and_touches_nothing_else(rot, interleaved):
    pk = require_gpu()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 11, 64, generator=g).to(torch.bfloat16).to(DEV)
    q, k = x[:, :6], x[:, 6:9]
    inv, _ = pk.rope_inv_freq(rot)
    pos = torch.arange(9, device=DEV) * 1000
    before = x.clone()
    qo, ko = pk.rope(q, k, pos, inv, interleaved=interleaved)
    assert torch.equal(x, before)
    a, b = pk.rope(q, k, pos, inv, interleaved=interleaved, q_out=q, k_out=k)
    assert a is q and b is k
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, 9:], before[:, 9:])


@pytest.mark.parametrize("dt", list(DT))
def test_rope_copies_the_other_dims_bit_exactly_whatever_they_hold(dt):
    pk = require_gpu()
    dt = DT[dt]
    raw = torch.int32 if dt == torch.float32 else torch.int16
    x = torch.zeros(2, 2, 64, dtype=dt, device=DEV)
    x[..., 16:] = torch.tensor([float("inf"), float("nan"), -0.0, 1e-7], dtype=dt, device=DEV).repeat(12)
    x.view(raw)[..., 60] = 0x7F83 if dt == torch.bfloat16 else 0x7C03 if dt == torch.float16 else 0x7F800003
    for inter, rot in [(False, 16), (True, 16), (True, 10), (False, 10), (True, 6), (False, 2)]:
        z = x.clone()
        z[..., rot:16] = float("nan")
        inv, _ = pk.rope_inv_freq(rot)
        y, _ = pk.rope(z, None, torch.tensor([3, 4], device=DEV), inv, interleaved=inter, mscale=2.0)
        assert torch.equal(y[..., rot:].view(raw), z[..., rot:].view(raw))
        assert torch.all(y[..., :rot] == 0)


def paged(nb, bs, hkv, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(nb, bs, hkv, d, generator=g).to(dt).to(DEV) for _ in range(2)]


STORES = [("f32", 4, 2, 64, 16, 64, False), ("bf16", 48, 8, 128, 16, 128, True), ("f16", 16, 16, 64, 256, 32, False),
          ("bf16", 6, 3, 128, 32, 36, False), ("f16", 2, 1, 64, 16, 20, True)]


@pytest.mark.parametrize("case", STORES, ids=["-".join(map(str, c)) for c in STORES])
def test_rope_store_paged(case):
    """q_out, the stored key (rotated) and value (bits), the slots, and not one other cache element."""
    pk = require_gpu()
    dt, hq, hkv, d, bs, rot, inter = case
    dt = DT[dt]
    nb = 40
    kc, vc = paged(nb, bs, hkv, d, dt, 4)
    k0, v0 = kc.clone(), vc.clone()
    # empty row, first token, block boundaries, a bad block, a context past the table, a negative one
    ctx = [0, 1, bs, bs + 1, 2 * bs + 3, 2, 3 * bs + 1, -4]
    B = len(ctx)
    tables = torch.arange(B * 3, dtype=torch.int32).view(B, 3) + 7
    tables[5, 0] = nb
    q, k, v = projected(B, hq, hkv, d, dt, 5)
    inv, m = pk.rope_inv_freq(rot, scaling="parts", factor=4.0)
    slots = torch.full((B,), 123, dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pk.rope_store_paged(q, k, v, tables.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), inv, kc, vc,
                              interleaved=inter, mscale=m, slot_mapping=slots, err=err)
    pos = [c - 1 for c in ctx]
    live = [i for i, c in enumerate(ctx) if c > 0]
    close(out[live], q[live], [pos[i] for i in live], inv.tolist(), inter, m)
    assert torch.all(out[[0, 7]] == 0)
    stored = [1, 2, 3, 4]
    want = [int(tables[i, pos[i] // bs]) * bs + pos[i] % bs if i in stored else -1 for i in range(B)]
    assert slots.tolist() == want
    assert err.item() == (pk.ERR_BLOCK_ID | pk.ERR_CONTEXT)
    at = torch.tensor([want[i] for i in stored], device=DEV)
    flat_k, flat_v = kc.view(-1, hkv, d), vc.view(-1, hkv, d)
    close(flat_k[at], k[stored], [pos[i] for i in stored], inv.tolist(), inter, m)
    assert torch.equal(flat_v[at], v[stored])
    flat_k[at] = k0.view(-1, hkv, d)[at]
    flat_v[at] = v0.view(-1, hkv, d)[at]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


@pytest.mark.parametrize("case", STORES, ids=["-".join(map(str, c)) for c in STORES])
def test_rope_store_prefill(case):
    """Ragged sequences (none, one and several new rows, cached prefixes), rows
    past the batch, and a sequence with more new rows than tokens."""
    pk = require_gpu()
    dt, hq, hkv, d, bs, rot, inter = case
    dt = DT[dt]
    nb = 64
    kc, vc = paged(nb, bs, hkv, d, dt, 6)
    k0, v0 = kc.clone(), vc.clone()
    qlen, klen = [3, 0, 1, bs + 2, 4], [3, 5, 2 * bs, bs + 7, 2]
    cq, ck = np.concatenate([[0], np.cumsum(qlen)]), np.concatenate([[0], np.cumsum(klen)])
    T, tail = int(cq[-1]), 2
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(7))[:len(qlen) * 3].to(torch.int32)
    tables = perm.view(len(qlen), 3)
    q, k, v = projected(T + tail, hq, hkv, d, dt, 8)
    inv, _ = pk.rope_inv_freq(rot)
    q_out = torch.full((T + tail, hq, d), 7.0, dtype=dt, device=DEV)
    slots = torch.full((T + tail,), 123, dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pk.rope_store_prefill(q, k, v, tables.to(DEV), torch.tensor(cq, dtype=torch.int32, device=DEV),
                                torch.tensor(ck, dtype=torch.int32, device=DEV), inv, kc, vc, interleaved=inter,
                                q_out=q_out, slot_mapping=slots, err=err)
    assert got is q_out and err.item() == pk.ERR_CONTEXT
    rows, pos, want = [], [], []
    for i in range(4):
        for j in range(qlen[i]):
            p = klen[i] - qlen[i] + j
            rows.append(int(cq[i]) + j)
            pos.append(p)
            want.append(int(tables[i, p // bs]) * bs + p % bs)
    close(q_out[rows], q[rows], pos, inv.tolist(), inter, 1.0)
    assert torch.all(q_out[T - 4:] == 7.0)                 # the bad sequence, and the rows behind the batch
    assert slots.tolist() == want + [-1] * (4 + tail)
    at = torch.tensor(want, device=DEV)
    close(kc.view(-1, hkv, d)[at], k[rows], pos, inv.tolist(), inter, 1.0)
    assert torch.equal(vc.view(-1, hkv, d)[at], v[rows])
    kc.view(-1, hkv, d)[at] = k0.view(-1, hkv, d)[at]
    vc.view(-1, hkv, d)[at] = v0.view(-1, hkv, d)[at]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_rope_store_into_one_layer_of_a_strided_cache():
    """Head-major and multi-layer caches: the strides of the views are followed."""
    pk = require_gpu()
    big = torch.zeros(2, 5, 3, 2, 16, 64, device=DEV)       # [kv, block, layer, head, row, dim]
    kc, vc = (big[i, :, 1].transpose(1, 2) for i in range(2))
    q, k, v = projected(2, 4, 2, 64, torch.float32, 9)
    inv, _ = pk.rope_inv_freq(64)
    ctx = torch.tensor([18, 3], dtype=torch.int32, device=DEV)
    tables = torch.tensor([[4, 2], [0, 1]], dtype=torch.int32, device=DEV)
    pk.rope_store_paged(q, k, v, tables, ctx, inv, kc, vc)
    assert torch.equal(vc[2, 1], v[0]) and torch.equal(vc[0, 2], v[1])
    close(torch.stack([kc[2, 1], kc[0, 2]]), k, [17, 2], inv.tolist(), False, 1.0)
    assert torch.count_nonzero(big).item() <= 4 * 2 * 64
    assert torch.count_nonzero(big[:, :, 0]).item() == 0 and torch.count_nonzero(big[:, :, 2]).item() == 0


def test_empty_calls():
    pk = require_gpu()
    inv, _ = pk.rope_inv_freq(64)
    q = torch.zeros(0, 4, 64, device=DEV)
    a, b = pk.rope(q, q, torch.zeros(0, dtype=torch.int64, device=DEV), inv)
    assert a.shape == (0, 4, 64) and b.shape == (0, 4, 64)
    kc, vc = paged(4, 16, 4, 64, torch.float32, 1)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    assert pk.rope_store_paged(q, q, q, t, z[:0], inv, kc, vc).shape == (0, 4, 64)
    assert pk.rope_store_prefill(q, q, q, t, z, z, inv, kc, vc).shape == (0, 4, 64)


def test_refusals():
    pk = require_gpu()
    inv, _ = pk.rope_inv_freq(64)
    q = torch.zeros(2, 4, 64, device=DEV)
    pos = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        pk.rope(q, q, pos.int(), inv)                       # int32 positions
    with pytest.raises(ValueError):
        pk.rope(q, q, pos[:1], inv)
    with pytest.raises(ValueError):
        pk.rope(q, q, pos, inv.float())
    with pytest.raises(ValueError):
        pk.rope(q, q, pos, inv.cpu())
    with pytest.raises(ValueError):
        pk.rope(q, q.half(), pos, inv)
    with pytest.raises(ValueError):
        pk.rope(q.transpose(1, 2), None, pos, inv)
    with pytest.raises(ValueError):
        pk.rope(q, None, pos, inv, q_out=q[:1])
    with pytest.raises(ValueError):
        pk.rope(q.cpu(), None, pos, inv)
    with pytest.raises(pk.PkvdError):
        pk.rope(torch.zeros(2, 4, 32, device=DEV), None, pos, inv)          # 64 rotated dims of 32
    with pytest.raises(TypeError):
        pk.rope(q.double(), None, pos, inv)
    with pytest.raises(ValueError):
        pk.rope_inv_freq(64, scaling="other")
    kc, vc = paged(4, 16, 4, 64, torch.float32, 1)
    tables = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    ctx = torch.ones(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        pk.rope_store_paged(q, q[:, :2], q, tables, ctx, inv, kc, vc)        # two key heads for a cache of four
    with pytest.raises(ValueError):
        pk.rope_store_paged(q, q, q, tables, ctx[:1], inv, kc, vc)
    with pytest.raises(ValueError):
        pk.rope_store_paged(q, q, q, tables.long(), ctx, inv, kc, vc)
    with pytest.raises(ValueError):
        pk.rope_store_paged(q, q, q, tables, ctx, inv, kc.half(), vc.half())
    with pytest.raises(ValueError):
        pk.rope_store_paged(q, q, q, tables, ctx, inv, kc, vc, err=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        pk.rope_store_prefill(q, q, q, tables, ctx, ctx[:1], inv, kc, vc)


def test_rope_on_another_stream_and_replayed_from_a_graph():
    pk = require_gpu()
    q, k, v = projected(4, 8, 2, 128, torch.bfloat16, 11)
    kc, vc = paged(8, 16, 2, 128, torch.bfloat16, 12)
    inv, _ = pk.rope_inv_freq(128)
    tables = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    ctx = torch.tensor([5, 17, 32, 1], dtype=torch.int32, device=DEV)
    want = pk.rope_store_paged(q, k, v, tables, ctx, inv, kc, vc)
    torch.cuda.synchronize()
    k1, v1 = kc.clone(), vc.clone()
    kc.zero_(), vc.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pk.rope_store_paged(q, k, v, tables, ctx, inv, kc, vc, stream=side)
    raw = pk.rope(q, k, (ctx - 1).long(), inv, stream=side.cuda_stream)[0]
    side.synchronize()
    at = [(0, 4), (3, 0), (5, 15), (6, 0)]
    for i, (b, r) in enumerate(at):
        assert torch.equal(kc[b, r], k1[b, r]) and torch.equal(vc[b, r], v[i])
    assert torch.equal(got, want) and torch.equal(raw, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.rope_store_paged(q, k, v, tables, ctx, inv, kc, vc, q_out=out)
    for shift in (1, 2):
        ctx += shift
        ctx.clamp_(max=32)
        g.replay()
        pos = (ctx - 1).tolist()
        close(out, q, pos, inv.tolist(), False, 1.0)
        for i, p in enumerate(pos):
            assert torch.equal(vc[int(tables[i, p // 16]), p % 16], v[i])
