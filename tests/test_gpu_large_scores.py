"""Attention with modified scores where the scores themselves are large: rows
all of whose scores lie thousands above or below zero, by their products or by
a distance bias.  Only differences within a row count, so the weights are as
those of any other row.  The products and their sums are whole numbers that
fp32 holds exactly: what is left of the oracle's bound are the roundings of
the score's own arithmetic."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_score_mod import DEV, DT, tolerances

pytestmark = pytest.mark.gpu


def place(keys, values, bs, dt, seed):
    """One sequence's rows [n, Hkv, D] in shuffled blocks: (K cache, V cache, table)."""
    n, hkv, d = keys.shape
    nb = -(-n // bs)
    order = torch.randperm(nb + 2, generator=torch.Generator().manual_seed(seed))
    kc, vc = (torch.full((nb + 2, bs, hkv, d), float("nan"), dtype=dt) for _ in range(2))
    for b in range(nb):
        m = min(bs, n - b * bs)
        kc[order[b], :m], vc[order[b], :m] = keys[b * bs:b * bs + m], values[b * bs:b * bs + m]
    return kc.to(DEV), vc.to(DEV), order[:nb].to(torch.int32).view(1, nb).to(DEV)


def rows_around(offset, n, qn, hq, hkv, d, dt, seed):
    """q [qn, hq, d], k, v [n, hkv, d] whose scores at scale 1/8 lie about `offset` (log2 units), some units apart."""
    g = torch.Generator().manual_seed(seed)
    raw = offset * 8 * np.log(2.0) / 128                # of the first component, eight bits of it
    step = 2.0 ** max(np.floor(np.log2(abs(raw))) - 7, 0)
    k = torch.zeros(n, hkv, d)
    k[:, :, 0] = abs(round(raw / step)) * step
    k[:, :, 1] = torch.randint(0, 25, (n, hkv), generator=g).float()
    q = torch.zeros(qn, hq, d)
    q[:, :, 0] = 128.0 if offset > 0 else -128.0
    q[:, :, 1] = torch.randint(0, 3, (qn, hq), generator=g).float()
    v = 1.0 + 0.25 * torch.randn(n, hkv, d, generator=g)
    return q.to(dt), k.to(dt), v.to(dt)


def check(got, q, k, v, positions, cap, slopes, prefix, tol):
    G = q.shape[1] // k.shape[1]
    qd, kd, vd = (x.double().numpy() for x in (q, k, v))
    for t, p in enumerate(positions):
        for h in range(q.shape[1]):
            want, bound = oracle.scores.attend(qd[t, h], kd[:, h // G], vd[:, h // G], p, 0.125, cap, slopes[h],
                                               prefix=prefix, dot_rounds=0, **tol)
            off = np.abs(got[t, h] - want)
            assert np.all(off <= bound), (t, h, float(off.max()), float(bound.max()))


OFFSETS = [1e3, -1e3, 5e3, -5e3, 9e3, -9e3, 2e4, -2e4, 5e4, -5e4]
MODES = {"prefix": (0.0, None), "cap": (2.0 ** 22, None), "bias": (0.0, 2.0 ** -6), "cap-bias": (2.0 ** 22, 2.0 ** -6)}


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
def test_prefill_rows_of_large_scores(dt, d, offset, mode):
    pk = require_gpu()
    dt, (cap, slope) = DT[dt], MODES[mode]
    n, qn, hq, hkv, bs = 300, 21, 4, 2, 16
    q, k, v = rows_around(offset, n, qn, hq, hkv, d, dt, 1)
    kc, vc, table = place(k, v, bs, dt, 2)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    slopes = np.zeros(hq) if slope is None else slope * np.arange(1, hq + 1)
    prefix = 40 if mode == "prefix" else 0
    for path in (1, 2, 3):
        out = pk.prefill_attention(
            q.to(DEV), kc, vc, table, cq, ck, qn, 0.125, path=path, softcap=cap,
            alibi_slopes=None if slope is None else torch.tensor(slopes, dtype=torch.float32, device=DEV),
            prefix_lens=torch.tensor([prefix], dtype=torch.int32, device=DEV) if prefix else None)
        check(out.double().cpu().numpy(), q, k, v, range(n - qn, n), cap, slopes, prefix, tolerances(dt, path != 1))


@pytest.mark.parametrize("cap", [0.0, 2.0 ** 22])
@pytest.mark.parametrize("slope", [-1.0, 1.0])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
def test_prefill_bias_over_a_long_row(dt, d, slope, cap):
    """8,000 keys that a slope of -1 puts up to 11,500 log2 units above the row's own key."""
    pk = require_gpu()
    dt = DT[dt]
    n, qn, hq, hkv, bs = 8000, 9, 2, 1, 64
    g = torch.Generator().manual_seed(3)
    q, k = torch.zeros(qn, hq, d), torch.zeros(n, hkv, d)
    q[:, :, 0], k[:, :, 0] = 1.0, torch.randint(0, 33, (n, hkv), generator=g).float()
    q, k = q.to(dt), k.to(dt)
    v = (1.0 + 0.25 * torch.randn(n, hkv, d, generator=g)).to(dt)
    kc, vc, table = place(k, v, bs, dt, 4)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    slopes = np.array([slope, slope / 4])
    for path in (1, 2, 3):
        out = pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, 0.125, path=path, softcap=cap,
                                   alibi_slopes=torch.tensor(slopes, dtype=torch.float32, device=DEV))
        check(out.double().cpu().numpy(), q, k, v, range(n - qn, n), cap, slopes, 0, tolerances(dt, path != 1))


@pytest.mark.parametrize("mode", ["cap", "bias", "cap-bias"])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128)])
def test_decode_rows_of_large_scores(dt, d, offset, mode):
    pk = require_gpu()
    dt, (cap, slope) = DT[dt], MODES[mode]
    n, hq, hkv, bs = 300, 16, 8, 16
    q, k, v = rows_around(offset, n, 1, hq, hkv, d, dt, 5)
    kc, vc, table = place(k, v, bs, dt, 6)
    slopes = np.zeros(hq) if slope is None else slope * np.arange(1, hq + 1)
    for path in (1, 2):
        out = pk.paged_decode_attention(
            q.to(DEV), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), n, 0.125, path=path,
            softcap=cap, alibi_slopes=None if slope is None else torch.tensor(slopes, dtype=torch.float32, device=DEV))
        check(out.double().cpu().numpy(), q, k, v, [n - 1], cap, slopes, 0, tolerances(dt, path != 1))


def steep_case(slope, n, qn, hq, hkv, d, dt, seed):
    """Scores of a few units under a slope so steep that a row's nearest key (a negative slope: its farthest) has all
    the weight."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(qn, hq, d, generator=g).to(dt)
    k = torch.randn(n, hkv, d, generator=g).to(dt)
    v = (1.0 + 0.25 * torch.randn(n, hkv, d, generator=g)).to(dt)
    return q, k, v, np.float32(slope) * np.ones(hq, dtype=np.float32)


def check_steep(got, v, hq, positions, prefix, steep, tol):
    """Each row is one key's values: its weight, rounded once, over a sum of that weight, rounded once more."""
    G, vd = hq // v.shape[1], v.double().numpy()
    for t, p in enumerate(positions):
        j = p if steep > 0 else 0 if p >= max(prefix - 1 - p, 0) else prefix - 1
        for h in range(hq):
            want = vd[j, h // G]
            bound = np.abs(want) * (tol["u_p"] + tol["eps"] / 2 + 2.0 ** -20)
            assert np.all(np.abs(got[t, h] - want) <= bound), (t, h, float(np.abs(got[t, h] - want).max()))


STEEP = [300.0, 1e4, 1e6, 1e9, 1e20]


@pytest.mark.parametrize("slope", [s * x for x in STEEP for s in (1, -1)])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
def test_prefill_of_steep_slopes(dt, d, slope):
    prefill_of_steep_slopes(dt, d, slope)


def prefill_of_steep_slopes(dt, d, slope):
    pk = require_gpu()
    dt = DT[dt]
    n, qn, hq, hkv, bs = 300, 41, 4, 2, 16
    q, k, v, slopes = steep_case(slope, n, qn, hq, hkv, d, dt, 7)
    kc, vc, table = place(k, v, bs, dt, 8)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    for prefix in (0, 100):
        for cap in (0.0, 50.0):
            for path in (1, 2, 3):
                out = pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, 0.125, path=path, softcap=cap,
                                           alibi_slopes=torch.from_numpy(slopes).to(DEV),
                                           prefix_lens=torch.tensor([prefix], dtype=torch.int32, device=DEV))
                check_steep(out.double().cpu().numpy(), v, hq, range(n - qn, n), prefix, slope,
                            tolerances(dt, path != 1))


@pytest.mark.parametrize("slope", [s * x for x in STEEP for s in (1, -1)])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128), ("f32", 64)])
def test_decode_of_steep_slopes(dt, d, slope):
    decode_of_steep_slopes(dt, d, slope)


def decode_of_steep_slopes(dt, d, slope):
    pk = require_gpu()
    dt = DT[dt]
    n, hq, hkv, bs = 300, 16, 8, 16
    q, k, v, slopes = steep_case(slope, n, 1, hq, hkv, d, dt, 9)
    kc, vc, table = place(k, v, bs, dt, 10)
    for path in (1,) if dt == torch.float32 else (1, 2):
        out = pk.paged_decode_attention(q.to(DEV), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), n,
                                        0.125, path=path, alibi_slopes=torch.from_numpy(slopes).to(DEV))
        check_steep(out.double().cpu().numpy(), v, hq, [n - 1], 0, slope, tolerances(dt, path != 1))


HUGE = [1e33, 1e36, 3e38]


@pytest.mark.parametrize("slope", [s * x for x in HUGE for s in (1, -1)])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128)])
def test_slopes_whose_bias_is_past_fp32(dt, d, slope):
    prefill_of_steep_slopes(dt, d, slope)
    decode_of_steep_slopes(dt, d, slope)


@pytest.mark.parametrize("large", [2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 28, -2.0 ** 25])
@pytest.mark.parametrize("d", [64, 128])
def test_f16_weights_of_scores_without_a_fraction(d, large):
    """Scores so large that fp32 holds them in steps of 2 to 32: what grows from tile to tile without a new reference
    still has to be a weight that f16 can hold."""
    pk = require_gpu()
    n, qn, hq, hkv, bs, dt = 1100, 5, 2, 1, 16, torch.float16
    g = torch.Generator().manual_seed(11)
    q, k = torch.zeros(qn, hq, d), torch.zeros(n, hkv, d)
    q[:, :, 0], k[:, :, 0] = large / 2.0 ** 13, 2.0 ** 15
    q[:, :, 1] = 8.0
    k[:, :, 1] = torch.randint(0, 8, (n, hkv), generator=g).float() + torch.arange(n, 0, -1)[:, None] // 32
    q, k = q.to(dt), k.to(dt)
    v = (1.0 + 0.25 * torch.randn(n, hkv, d, generator=g)).to(dt)
    kc, vc, table = place(k, v, bs, dt, 12)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    scale = 0.25 / np.log2(np.e)                       # the first component comes to `large` in log2 units
    for path in (1, 2, 3):
        out = pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, float(scale), path=path,
                                   prefix_lens=torch.tensor([3], dtype=torch.int32, device=DEV)).double().cpu().numpy()
        lo, hi = float(v.min()), float(v.max())
        assert np.all(out >= lo - abs(lo) * 2.0 ** -9) and np.all(out <= hi + abs(hi) * 2.0 ** -9), path


@pytest.mark.parametrize("steps", [9.5, 1.49, 0.3])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_small_weights_beside_one_whose_value_is_zero(dt, steps):
    """All but one key of a row have `steps` of f16's smallest step (2^-24) of the largest one's weight, and that one's
    values are zero: the small weights are the whole result."""
    pk = require_gpu()
    n, qn, hq, hkv, d, bs, dt = 3000, 5, 8, 8, 64, 64, DT[dt]
    g = torch.Generator().manual_seed(15)
    k = torch.zeros(n, hkv, d)
    k[n - 20, :, 0] = 1.0
    q = torch.zeros(qn, hq, d)
    q[:, :, 0] = 1.0
    k, q = k.to(dt), q.to(dt)
    v = 64 * (1.0 + 0.25 * torch.randn(n, hkv, d, generator=g))
    v[n - 20] = 0.0
    v = v.to(dt)
    scale = float(-np.log(steps * 2.0 ** -24))
    kc, vc, table = place(k, v, bs, dt, 16)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    zero = torch.zeros(hq, device=DEV)
    # the tcgen05 path's reference may lag 2^8 behind the largest weight, which leaves it seven bits below 2^-14
    got = [pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, scale, path=path, alibi_slopes=zero)[qn - 1]
           for path in ((2, 3) if dt == torch.bfloat16 or steps > 8 else (2,))]
    got.append(pk.paged_decode_attention(q[:1].to(DEV), kc, vc, table, ck[1:], n, scale, path=2, alibi_slopes=zero)[0])
    for h in range(hq):
        want, bound = oracle.scores.attend(q[0, h].double().numpy(), k[:, h].double().numpy(), v[:, h].double().numpy(),
                                           n - 1, scale, dot_rounds=0, **tolerances(dt, True))
        for i, o in enumerate(got):
            off = np.abs(o[h].double().cpu().numpy() - want)
            assert np.all(off <= bound), (i, h, float((off / bound).max()))
