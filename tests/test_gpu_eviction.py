"""Counted attention weights, which positions stay, and the moves of cached rows."""
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


# ------------------------------------------------------------------ weights
def run_weights(pk, case, ctx, mod=(0.0, None, 0), heads=None, seed=0, every=1, slack=0):
    dt, hq, hkv, d, bs, path = case
    dt = DT[dt]
    cap, kind, window = mod
    heads = hkv if heads is None else heads
    group = hq // hkv
    kc, vc, tables, rows = cache_of(ctx, hkv, d, bs, dt, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (3 * torch.randn(len(ctx), hq, d, generator=g)).to(dt)
    dev_slopes, slopes = slopes_for(hq, kind)
    scale, err, most = d ** -0.5, torch.zeros(1, dtype=torch.int32, device=DEV), max(max(ctx), 1)
    before = torch.rand(len(ctx), heads, most + slack, generator=g)
    dev = before.to(DEV)
    out, after = pk.paged_decode_attention_weights(q.to(DEV), kc, vc, tables, ints(ctx), most, scale, dev, window=window,
                                                   softcap=cap, alibi_slopes=dev_slopes, err=err, path=path)
    assert err.item() == 0 and after is dev
    got, added = out.double().cpu().numpy(), after.double().cpu().numpy()
    tensor = dt != torch.float32 and path != 1 and hkv in (8, 16)
    tol = tolerances(dt, tensor)
    for i, n in enumerate(ctx):
        assert torch.equal(after[i, :, n:].cpu(), before[i, :, n:])          # not these
        if n == 0:
            assert np.all(got[i] == 0)
            continue
        for h in range(0, hq, every):
            k, v = (x[:, h // group] for x in rows[i])
            want, bound = oracle.scores.attend(q[i, h].double().numpy(), k, v, n - 1, scale, cap, slopes[h], window, **tol)
            assert np.all(np.abs(got[i, h] - want) <= bound), (i, h)
        for r in range(heads):
            mine = range(hq) if heads == 1 else range(r * group, (r + 1) * group)
            total, bound = before[i, r, :n].double().numpy(), 0.0
            for h in mine:
                w, b = oracle.drafts.given(q[i, h].double().numpy(), rows[i][0][:, h // group], n, scale, cap, slopes[h], window)
                total, bound = total + w, bound + b
            # each of the sums (heads, and what was there) is rounded once, at no more than the result
            bound = bound + (len(mine) + 1) * 2.0 ** -24 * total
            off = np.abs(added[i, r, :n] - total)
            assert np.all(off <= bound), (i, r, float((off - bound).max()))
    return out, after


DECODE = [  # dtype, hq, hkv, d, bs, path
    ("f32", 4, 2, 64, 16, 0), ("f32", 8, 8, 64, 32, 0), ("f32", 15, 5, 64, 16, 0), ("bf16", 48, 8, 128, 16, 0),
    ("bf16", 48, 8, 128, 16, 1), ("f16", 16, 16, 64, 256, 0), ("f16", 64, 8, 64, 16, 2), ("f16", 3, 1, 128, 64, 0),
    ("bf16", 12, 6, 64, 16, 0), ("f16", 128, 16, 64, 16, 1),
]
MODS = [(0.0, None, 0), (5.0, None, 0), (2.0, "mixed", 0), (0.0, "geometric", 37), (0.0, None, 1)]


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c)))
def test_weights(case, mod):
    pk = require_gpu()
    run_weights(pk, case, [1, 0, 16, 17, 333, 50, 700], mod, every=5 if case[1] > 8 else 1)


@pytest.mark.parametrize("case", DECODE[:6], ids=lambda c: "-".join(map(str, c)))
def test_one_row_of_weights_for_all_heads(case):
    pk = require_gpu()
    run_weights(pk, case, [5, 300, 0, 1025], (0.0, "geometric", 0), heads=1, every=7, slack=5)


def test_weights_of_long_rows_and_many():
    pk = require_gpu()
    run_weights(pk, ("bf16", 16, 8, 128, 16, 0), [20001], seed=3, every=5)
    run_weights(pk, ("f32", 2, 1, 64, 64, 0), [9000, 2], seed=4)
    run_weights(pk, ("f16", 8, 8, 64, 16, 0), np.random.default_rng(5).integers(0, 60, 400).tolist(), seed=5, every=8)


def test_weights_agree_with_the_plain_call_and_add_up():
    """The output is the plain call's within the last rounding, a step's weights sum to its heads, steps add up."""
    pk = require_gpu()
    ctx = [40, 333, 1, 0]
    kc, vc, tables, _ = cache_of(ctx, 8, 128, 16, torch.bfloat16, 6)
    q = torch.randn(4, 24, 128, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
    args = (q, kc, vc, tables, ints(ctx), 333, 0.09)
    weights = torch.zeros(4, 8, 400, device=DEV)
    out, _ = pk.paged_decode_attention_weights(*args, weights)
    plain = pk.paged_decode_attention(*args)
    # the same products and weights; the sums' order is the same too
    assert torch.allclose(out.float(), plain.float(), rtol=2.0 ** -7, atol=2.0 ** -20)
    sums = weights.double().sum(dim=2).cpu()
    assert torch.allclose(sums[:3], torch.full((3, 8), 3.0, dtype=torch.float64), atol=3 * 333 * 2.0 ** -22)
    assert torch.all(sums[3] == 0) and torch.all(weights[:, :, 333:] == 0)
    once = weights.clone()
    elsewhere = torch.full_like(weights, -1.0)
    pk.paged_decode_attention_weights(*args, once, weights_out=elsewhere)
    assert torch.equal(weights, once)                        # only read
    pk.paged_decode_attention_weights(*args, weights)
    assert torch.equal(weights[1, :, :333], elsewhere[1, :, :333]) and torch.all(elsewhere[1, :, 333:] == -1)
    for _ in range(3):                                       # the same bits in every run
        again = once.clone()
        pk.paged_decode_attention_weights(*args, again)
        assert torch.equal(again, weights)


def test_weights_with_bad_device_data():
    pk = require_gpu()
    ctx = [200, 100]
    kc, vc, tables, _ = cache_of(ctx, 8, 64, 16, torch.float16, 8)
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(9)).to(torch.float16).to(DEV)
    for path in (1, 2):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        t = tables.clone()
        t[0, 3] = -5                                         # positions 48 .. 63
        weights = torch.zeros(2, 8, 200, device=DEV)
        pk.paged_decode_attention_weights(q, kc, vc, t, ints(ctx), 200, 0.1, weights, err=err, path=path)
        assert err.item() == pk.ERR_BLOCK_ID
        assert torch.all(weights[0, :, 48:64] == 0) and torch.all(weights[0, :, :48] > 0) and torch.all(weights[0, :, 64:] > 0)
        err.zero_()
        weights.zero_()
        pk.paged_decode_attention_weights(q, kc, vc, tables, ints([-3, 100]), 200, 0.1, weights, err=err, path=path)
        assert err.item() == pk.ERR_CONTEXT and torch.all(weights[0] == 0) and torch.all(weights[1, :, :100] > 0)
        err.zero_()
        long = torch.zeros(2, 8, 200, device=DEV)
        pk.paged_decode_attention_weights(q, kc, vc, tables, ints([200, 150]), 100, 0.1, long, err=err, path=path)
        assert err.item() == pk.ERR_CONTEXT and torch.all(long[:, :, 100:] == 0)      # cut to the bound


def test_weights_captured_and_on_two_streams():
    pk = require_gpu()
    ctx = [300, 77, 1000]
    kc, vc, tables, _ = cache_of(ctx, 8, 128, 32, torch.bfloat16, 10)
    q = torch.randn(3, 64, 128, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).to(DEV)
    args = (q, kc, vc, tables, ints(ctx), 1000, 0.09)
    ref = torch.zeros(3, 8, 1000, device=DEV)
    out, _ = pk.paged_decode_attention_weights(*args, ref)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    x, y = torch.zeros_like(ref), torch.zeros_like(ref)
    torch.cuda.synchronize()
    a, _ = pk.paged_decode_attention_weights(*args, x, stream=s)
    b, _ = pk.paged_decode_attention_weights(*args, y, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(x, ref) and torch.equal(y, ref) and torch.equal(a, out) and torch.equal(b, out)
    n = pk.decode_weights_workspace_bytes(3, 64, 128, 1000)
    ws, o = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(out)
    pk.paged_decode_attention_weights(*args, x, workspace=ws, out=o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.paged_decode_attention_weights(*args, x, workspace=ws, out=o)
    x.zero_()
    ws.fill_(0xff)
    o.zero_()
    graph.replay()
    assert torch.equal(x, ref) and torch.equal(o, out)


# ------------------------------------------------------------------- select
def run_select(pk, w, ctx, keep, sink, recent, in_place=False, err=None):
    dev = w.to(DEV)
    held = dev if in_place else torch.full_like(dev, 9.0)
    pos, counts = pk.evict_select(dev, ints(ctx), keep, sink=sink, recent=recent, weights_out=held, err=err)
    if not in_place:
        assert torch.equal(dev.cpu().view(torch.int32), w.view(torch.int32))
    pos, held, a = pos.cpu(), held.cpu(), w.numpy()
    for i, n in enumerate(ctx):
        assert counts[i].item() == min(n, keep)
        for h in range(w.shape[1]):
            want = oracle.drafts.stays(a[i, h], n, keep, sink, recent)
            assert pos[i, h].tolist() == want + [-1] * (keep - len(want)), (i, h)
            line = held[i, h]
            assert torch.equal(line[:len(want)].view(torch.int32), w[i, h, want].view(torch.int32))
            assert torch.all(line[len(want):] == 0)
    return pos


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (24, 4, 8), (24, 0, 24), (24, 24, 0), (24, 12, 12),
                                              (200, 4, 50), (5000, 4, 100)])
def test_select(keep, sink, recent, in_place):
    pk = require_gpu()
    ctx = [0, 1, 2, 24, 25, 26, 199, 200, 201, 1024, 1025, 3000]
    g = torch.Generator().manual_seed(keep)
    w = torch.empty(len(ctx), 2, 3000).exponential_(1.0, generator=g) ** 4
    run_select(pk, w, ctx, keep, sink, recent, in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "signed", "tiny", "huge", "special"])
def test_select_values(kind):
    """Ties by the thousand, zeros of both signs, subnormals, infinities and NaN: the order of the numbers, then of the positions."""
    pk = require_gpu()
    g = torch.Generator().manual_seed(3)
    n = 2500
    w = torch.rand(2, 3, n, generator=g)
    if kind == "equal":
        w.fill_(0.3)
    elif kind == "zeros":
        w = torch.where(w < 0.5, torch.tensor(0.0), torch.tensor(-0.0))
    elif kind == "few":
        w = torch.round(w * 4) / 4
    elif kind == "signed":
        w = w - 0.5
    elif kind == "tiny":
        w = torch.round(w * 40) * 2.0 ** -149
    elif kind == "huge":
        w = w * 3e38
    else:
        w = torch.round(w * 20)
        for value, at in ((float("inf"), 3), (float("-inf"), 7), (float("nan"), 11)):
            w[w == at] = value
    for keep, sink, recent in ((100, 3, 20), (1500, 0, 0), (2499, 5, 5)):
        run_select(pk, w, [n, 2200], keep, sink, recent)


@pytest.mark.parametrize("near", [1, 255, 256, 257, 512])
@pytest.mark.parametrize("keep", [1, 100, 255, 300])
def test_select_crowded_weights(near, keep):
    """Many weights that differ in late bits alone, in one stretch of a row: as many as are kept aside, and more."""
    pk = require_gpu()
    g = torch.Generator().manual_seed(near)
    w = 0.1 * torch.rand(2, 2, 8192, generator=g)
    w[:, :, :near] = 1 + 0.25 * torch.rand(2, 2, near, generator=g)
    w[1, :, 4096:4096 + near] = 1 + 0.25 * torch.rand(2, near, generator=g)
    w[:, 1, 5000:5003] = 7.0
    run_select(pk, w, [8192, 8192], keep, 0, 0)
    run_select(pk, w, [8192, 8100], keep, 0, 0, in_place=True)


@pytest.mark.parametrize("seqs", [2, 45, 256, 257])
def test_select_of_many_rows(seqs):
    """More rows than run at once, of all lengths, equal and none among them: every row in its own place."""
    pk = require_gpu()
    rng = np.random.default_rng(seqs)
    heads = 200 if seqs == 2 else 8 if seqs == 45 else 2
    ctx = rng.choice([0, 1, 17, 64, 65, 100, 199, 200], seqs).tolist()
    w = torch.rand(seqs, heads, 200, generator=torch.Generator().manual_seed(seqs))
    run_select(pk, w, ctx, 60, 3, 10)
    run_select(pk, w, ctx[::-1], 60, 3, 10, in_place=True)


@pytest.mark.parametrize("more", [-1, 0, 1, 40])
@pytest.mark.parametrize("sink", [0, 1, 2, 3, 4])
def test_select_in_place_where_memory_on_the_chip_ends(sink, more):
    """Rows about as long as what a row's kernel holds, beginning at every offset from a boundary of 16 bytes."""
    pk = require_gpu()
    n = 44 * 512 + sink + more
    w = torch.empty(1, 2, n).exponential_(1.0, generator=torch.Generator().manual_seed(sink))
    run_select(pk, w, [n], 20000, sink, 5, in_place=True)
    run_select(pk, w, [n - 3], 300, sink, 0)


def test_select_long_rows_of_other_strides():
    """Rows longer than one pass over shared memory would hold, inside a wider buffer at an odd offset."""
    pk = require_gpu()
    g = torch.Generator().manual_seed(4)
    n = 70001
    w = torch.empty(2, 2, n).exponential_(1.0, generator=g)
    run_select(pk, w, [n, 40000], 4000, 4, 300)
    run_select(pk, w, [n, 66000], 65000, 4, 300, in_place=True)
    wide = torch.full((2, 2, n + 7), 5.0, device=DEV)
    wide[:, :, 3:3 + n] = w.to(DEV)
    pos, _ = pk.evict_select(wide[:, :, 3:3 + n], ints([n, 40000]), 4000, sink=4, recent=300, weights_out=wide[:, :, 3:3 + n])
    ref, _ = pk.evict_select(w.to(DEV), ints([n, 40000]), 4000, sink=4, recent=300)
    assert torch.equal(pos, ref) and torch.all(wide[:, :, :3] == 5) and torch.all(wide[:, :, 3 + n:] == 5)


def test_select_clamps_lengths():
    pk = require_gpu()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.rand(3, 1, 50, device=DEV)
    pos, counts = pk.evict_select(w, ints([-4, 60, 50]), 10, err=err)
    assert err.item() == pk.ERR_CONTEXT and counts.tolist() == [0, 10, 10]
    want, _ = pk.evict_select(w, ints([0, 50, 50]), 10, err=err)
    assert torch.equal(pos, want)


def test_select_captured():
    pk = require_gpu()
    w = torch.rand(4, 8, 2000, device=DEV)
    ctx = ints([2000, 5, 1999, 600])
    ref = pk.evict_select(w, ctx, 500, sink=2, recent=9)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pk.evict_select(w, ctx, 500, sink=2, recent=9)
    for _ in range(2):
        got[0].fill_(7)
        graph.replay()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ------------------------------------------------------------------ compact
def a_cache(nb, bs, hkv, d, dt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    raw = lambda: torch.randint(-2 ** 15, 2 ** 15, (nb, bs, hkv, d * torch.finfo(dt).bits // 16), generator=g, device=DEV,
                                dtype=torch.int16).view(dt)        # any bits, NaN among them
    return raw(), raw()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def moved(cache, tables, new_tables, positions, counts, first, bs):
    """The rows that a call has to leave, by its definition."""
    a = bits(cache)
    out = a.copy()
    for i, n in enumerate(counts):
        for h in range(a.shape[2]):
            row = positions[i] if positions.ndim == 2 else positions[i, h % positions.shape[1]]
            for r in range(n):
                s, t = int(row[r]), first[i] + r
                out[new_tables[i][t // bs], t % bs, h] = a[tables[i][s // bs], s % bs, h]
    return out


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("case", [("bf16", 8, 128, 16), ("f32", 3, 128, 32), ("f16", 1, 64, 256), ("f32", 2, 64, 1), ("bf16", 16, 64, 8)],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("heads", ["alike", "one", "own"])
def test_compact(case, heads, fresh):
    pk = require_gpu()
    dt, hkv, d, bs = case
    rng = np.random.default_rng(bs + hkv)
    lens, first = [700, 1, 300, 64, 129, 0], [0, 0, 37, 60, 129, 0]
    keep = [600, 1, 200, 3, 0, 0]
    need = [-(-n // bs) for n in lens]
    nb = 2 * sum(need) + 3
    order = rng.permutation(nb)
    cut = np.split(order[:2 * sum(need)], np.cumsum(need + need)[:-1])
    width = max(need)
    table = lambda part: np.array([list(x) + [-1] * (width - len(x)) for x in part])
    old, new = table(cut[:6]), table(cut[6:]) if fresh else None
    lists = 1 if heads != "own" else hkv
    pos = np.full((6, lists, max(keep) + 2), -1)
    for i, k in enumerate(keep):
        for h in range(lists):
            pos[i, h, :k] = np.sort(rng.choice(np.arange(first[i], lens[i]), k, replace=False)) if k else []
    if heads == "alike":
        pos = pos[:, 0]
    kc, vc = a_cache(nb, bs, hkv, d, DT[dt], 1)
    want = [moved(x, old, new if fresh else old, pos, keep, first, bs) for x in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.compact_cache(kc, vc, ints(old.tolist()), ints(pos.tolist()), ints(keep), first=ints(first),
                     new_tables=ints(new.tolist()) if fresh else None, err=err)
    assert err.item() == 0
    for x, y in zip((kc, vc), want):
        assert np.array_equal(bits(x), y)


def test_compact_in_any_order_and_with_repeats():
    """In place only positions[r] >= first + r counts; into other blocks any list does."""
    pk = require_gpu()
    rng = np.random.default_rng(3)
    n, bs, keep = 2000, 16, 900
    table = rng.permutation(2 * n // bs)[:n // bs][None]
    other = np.setdiff1d(np.arange(2 * n // bs), table)[None]
    pos = np.array([[int(rng.integers(r, n)) for r in range(keep)]])
    pos[0, 5:9] = 1999
    for new in (None, other):
        if new is not None:
            pos = rng.integers(0, n, (1, keep))
        kc, vc = a_cache(2 * n // bs, bs, 2, 64, torch.float16, 2)
        want = [moved(x, table, table if new is None else new, pos, [keep], [0], bs) for x in (kc, vc)]
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pk.compact_cache(kc, vc, ints(table.tolist()), ints(pos.tolist()), ints([keep]),
                         new_tables=None if new is None else ints(new.tolist()), err=err)
        assert err.item() == 0 and all(np.array_equal(bits(x), y) for x, y in zip((kc, vc), want))


def test_compact_errors_in_device_data():
    pk = require_gpu()
    kc, vc = a_cache(8, 16, 2, 64, torch.float16, 3)
    keep = [x.clone() for x in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = ints([[3, 1, 5]])
    same = lambda: all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((kc, vc), keep))

    def call(pos, counts=None, first=None, tables=table, new=None):
        err.zero_()
        p = ints([pos])
        pk.compact_cache(kc, vc, tables, p, ints([len(pos) if counts is None else counts]),
                         first=None if first is None else ints([first]), new_tables=new, err=err)
        return err.item()
    assert call([48]) == pk.ERR_CONTEXT and same()                       # past the table
    assert call([-1]) == pk.ERR_CONTEXT and same()
    assert call([1, 0]) == pk.ERR_CONTEXT                                # below its place, in place: that row is not copied
    kc.copy_(keep[0]), vc.copy_(keep[1])
    assert call([0, 1], counts=-1) == pk.ERR_CONTEXT and same()
    assert call([0, 1], counts=9) == pk.ERR_CONTEXT and same()
    assert call([5], first=-2) == pk.ERR_CONTEXT and same()
    assert call([20], tables=ints([[3, 8, 5]])) == pk.ERR_BLOCK_ID and same()
    assert call([20], new=ints([[-1, 2, 4]])) == pk.ERR_BLOCK_ID and same()
    assert call([20], first=47, new=ints([[0, 2]])) == pk.ERR_CONTEXT and same()


def test_compact_blocks_past_32_bit_offsets():
    pk = require_gpu()
    hkv, d, bs = 8, 128, 16
    nb = (1 << 32) // (bs * hkv * d * 2) + 300
    kc, vc = (torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rows = torch.randn(2, bs, hkv, d, device=DEV).to(torch.bfloat16)
    kc[nb - 2:], vc[nb - 2:] = rows, -rows
    pk.compact_cache(kc, vc, ints([[nb - 1, nb - 2]]), ints([[3, 20, 30]]), ints([3]), new_tables=ints([[nb - 7]]))
    want = torch.stack([rows[1, 3], rows[0, 4], rows[0, 14]])
    assert torch.equal(kc[nb - 7, :3], want) and torch.equal(vc[nb - 7, :3], -want)
    assert not kc[:nb - 7].any() and not kc[nb - 6:nb - 2].any()
