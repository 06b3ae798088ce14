"""Attention over the paged cache with capped, biased and prefix-open scores:
decode and prefill, every path, against the float64 oracle within its counted
bound."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def tolerances(dt, tensor_cores):
    """Half a step for the weights where they are rounded to the cache's type, and for the output."""
    return dict(u_p=EPS[dt] / 2 if tensor_cores else 0.0, eps=EPS[dt], tiny=2.0 ** -24 if dt == torch.float16 else 0.0)


def cache_of(klens, hkv, d, bs, dt, seed, spare=3):
    """Caches whose unused rows and blocks hold NaN, tables with -1 past each row's blocks."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in klens]
    nb, width = sum(need) + spare, max(max(need), 1) + 1
    kc, vc = (torch.full((nb, bs, hkv, d), float("nan"), dtype=dt) for _ in range(2))
    tables = torch.full((len(klens), width), -1, dtype=torch.int32)
    order = torch.randperm(nb, generator=g)
    rows, at = [], 0
    for i, n in enumerate(klens):
        k, v = (torch.randn(n, hkv, d, generator=g).to(dt) for _ in range(2))
        for b in range(need[i]):
            blk = int(order[at])
            at += 1
            tables[i, b] = blk
            m = min(bs, n - b * bs)
            kc[blk, :m], vc[blk, :m] = k[b * bs:b * bs + m], v[b * bs:b * bs + m]
        rows.append((k.double().numpy(), v.double().numpy()))
    return kc.to(DEV), vc.to(DEV), tables.to(DEV), rows


def slopes_for(hq, kind):
    if kind is None:
        return None, np.zeros(hq)
    s = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])
    if kind == "mixed":                       # zero, negative and steep ones among them
        s[::3] = 0.0
        s[1::4] *= -0.05
        s[2::5] = 3.0
    return s.to(DEV), s.double().numpy()


DECODE = [  # dtype, hq, hkv, d, bs, path
    ("f32", 4, 2, 64, 16, 0), ("f32", 8, 8, 64, 32, 0), ("f32", 15, 5, 64, 16, 0),
    ("bf16", 48, 8, 128, 16, 0), ("bf16", 48, 8, 128, 16, 1), ("f16", 16, 16, 64, 256, 0), ("f16", 128, 16, 64, 16, 0),
    ("f16", 3, 1, 128, 64, 0), ("bf16", 64, 8, 64, 16, 2), ("bf16", 12, 6, 64, 16, 0),
]
MODS = [(5.0, None, 0), (0.0, "geometric", 0), (2.0, "mixed", 0), (30.0, "geometric", 37), (1e5, "mixed", 1)]


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c)))
def test_decode(case, mod):
    pk = require_gpu()
    dt, hq, hkv, d, bs, path = case
    dt = DT[dt]
    cap, kind, window = mod
    ctx = [1, 0, 16, 17, 333, 50, 700]
    kc, vc, tables, rows = cache_of(ctx, hkv, d, bs, dt, 1)
    q = (3 * torch.randn(len(ctx), hq, d, generator=torch.Generator().manual_seed(2))).to(dt)
    dev_slopes, slopes = slopes_for(hq, kind)
    scale, err = d ** -0.5, torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pk.paged_decode_attention(q.to(DEV), kc, vc, tables, torch.tensor(ctx, dtype=torch.int32, device=DEV),
                                    max(ctx), scale, window=window, softcap=cap, alibi_slopes=dev_slopes, err=err,
                                    path=path)
    assert err.item() == 0
    got = out.double().cpu().numpy()
    tensor = dt != torch.float32 and path != 1 and hkv in (8, 16)
    tol = tolerances(dt, tensor)
    for i, n in enumerate(ctx):
        for h in range(hq):
            k, v = (x[:, h // (hq // hkv)] for x in rows[i])
            want, bound = oracle.scores.attend(q[i, h].double().numpy(), k, v, n - 1, scale, cap, slopes[h], window,
                                               **tol)
            off = np.abs(got[i, h] - want)
            assert np.all(off <= bound), (i, h, float((off - bound).max()))


PREFILL = [  # dtype, hq, hkv, d, bs, path
    ("bf16", 48, 8, 128, 16, 3), ("f16", 16, 16, 64, 256, 3), ("bf16", 8, 1, 64, 32, 3), ("f16", 6, 2, 128, 128, 3),
    ("bf16", 48, 8, 128, 16, 2), ("f16", 4, 4, 64, 64, 2), ("f32", 4, 2, 64, 16, 1), ("bf16", 6, 2, 128, 16, 1),
]
PREFILL_MODS = [  # cap, slopes, window, prefix lengths
    (5.0, None, 0, None), (0.0, "geometric", 0, None), (0.0, None, 0, [0, 1, 200, 40, 999]),
    (2.0, "mixed", 19, [5, 0, 130, 64, 10]), (30.0, "geometric", 0, [33, -4, 129, 128, 0]), (1e5, "mixed", 150, None),
]


@pytest.mark.parametrize("mod", PREFILL_MODS, ids=lambda m: "-".join(str(x).replace(" ", "") for x in m))
@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(map(str, c)))
def test_prefill(case, mod):
    pk = require_gpu()
    dt, hq, hkv, d, bs, path = case
    dt = DT[dt]
    cap, kind, window, prefix = mod
    qlen, klen = [70, 1, 45, 0, 3], [70, 131, 301, 40, 257]
    kc, vc, tables, rows = cache_of(klen, hkv, d, bs, dt, 3)
    T, tail = sum(qlen), 2
    q = (3 * torch.randn(T + tail, hq, d, generator=torch.Generator().manual_seed(4))).to(dt)
    cq, ck = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (qlen, klen))
    dev_slopes, slopes = slopes_for(hq, kind)
    scale, err = d ** -0.5, torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((T + tail, hq, d), 7.0, dtype=dt, device=DEV)
    pl = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, max(qlen), scale, window=window, out=out, err=err,
                         path=path, softcap=cap, alibi_slopes=dev_slopes, prefix_lens=pl)
    assert err.item() == 0
    assert torch.all(out[T:] == 7.0)
    got = out.double().cpu().numpy()
    tol = tolerances(dt, path != 1)
    t = 0
    for i, n in enumerate(klen):
        open_to = min(max(prefix[i], 0), n) if prefix else 0
        for j in range(qlen[i]):
            p = n - qlen[i] + j
            for h in range(hq):
                if (j * hq + h) % 5 and hq > 8:         # every fifth (row, head) of the wide layouts
                    continue
                k, v = (x[:, h // (hq // hkv)] for x in rows[i])
                want, bound = oracle.scores.attend(q[t, h].double().numpy(), k, v, p, scale, cap, slopes[h], window,
                                                   open_to, **tol)
                off = np.abs(got[t, h] - want)
                assert np.all(off <= bound), (i, j, h, float((off - bound).max()))
            t += 1


@pytest.mark.parametrize("path", [1, 2, 3])
def test_modifiers_that_do_nothing_agree_with_the_plain_call(path):
    """A zero slope array, an open prefix of nothing: the plain result within one rounding of the output."""
    pk = require_gpu()
    klen, qlen = [90, 200], [90, 30]
    kc, vc, tables, _ = cache_of(klen, 8, 64, 16, torch.bfloat16, 5)
    q = torch.randn(120, 8, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    cq, ck = (torch.tensor([0, x[0], sum(x)], dtype=torch.int32, device=DEV) for x in (qlen, klen))
    plain = pk.prefill_attention(q, kc, vc, tables, cq, ck, 90, 0.125, path=path)
    z = torch.zeros(8, device=DEV)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    got = pk.prefill_attention(q, kc, vc, tables, cq, ck, 90, 0.125, path=path, alibi_slopes=z, prefix_lens=none)
    assert torch.allclose(got.float(), plain.float(), rtol=2.0 ** -6, atol=2.0 ** -8)
    ctx = torch.tensor(klen, dtype=torch.int32, device=DEV)
    if path != 3:
        a = pk.paged_decode_attention(q[:2], kc, vc, tables, ctx, 200, 0.125, path=path)
        b = pk.paged_decode_attention(q[:2], kc, vc, tables, ctx, 200, 0.125, path=path, alibi_slopes=z)
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_bad_blocks_and_lengths_are_flagged():
    pk = require_gpu()
    kc, vc, tables, _ = cache_of([40, 20], 8, 64, 16, torch.float16, 7)
    q = torch.ones(2, 8, 64, dtype=torch.float16, device=DEV)
    ctx = torch.tensor([40, 20], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = tables.clone()
    bad[0, 1] = kc.shape[0]
    for path in (1, 2):
        err.zero_()
        out = pk.paged_decode_attention(q, kc, vc, bad, ctx, 40, 0.1, softcap=9.0, err=err, path=path)
        good = pk.paged_decode_attention(q, kc, vc, tables, ctx, 40, 0.1, softcap=9.0, path=path)
        assert err.item() == pk.ERR_BLOCK_ID and torch.equal(out[1], good[1])
    err.zero_()
    pk.paged_decode_attention(q, kc, vc, tables, ctx, 30, 0.1, softcap=9.0, err=err)
    assert err.item() == pk.ERR_CONTEXT
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 2], [0, 40, 60]))
    pre = torch.tensor([40, 20], dtype=torch.int32, device=DEV)
    for path in (1, 2, 3):
        err.zero_()
        pk.prefill_attention(q, kc, vc, bad, cq, ck, 1, 0.1, softcap=9.0, prefix_lens=pre, err=err, path=path)
        assert err.item() == pk.ERR_BLOCK_ID
        err.zero_()
        out = torch.full_like(q, 7.0)
        pk.prefill_attention(q, kc, vc, tables, cq.flip(0).contiguous() * 0 + cq, ck * 0, 1, 0.1, softcap=9.0,
                             prefix_lens=pre, err=err, path=path, out=out)
        assert err.item() == pk.ERR_CONTEXT and torch.all(out == 7.0)     # more rows than tokens


def test_refusals():
    pk = require_gpu()
    kc, vc, tables, _ = cache_of([40, 20], 8, 64, 16, torch.float16, 8)
    q = torch.ones(2, 8, 64, dtype=torch.float16, device=DEV)
    ctx = torch.tensor([40, 20], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    s = torch.ones(8, device=DEV)
    call = lambda **kw: pk.paged_decode_attention(kw.pop("q", q), kc, vc, tables, kw.pop("ctx", ctx), 40, 0.1, **kw)
    pre = lambda **kw: pk.prefill_attention(q, kc, vc, tables, cu, kw.pop("ck", cu), 1, 0.1, **kw)
    for bad in (dict(alibi_slopes=s[:7]), dict(alibi_slopes=s.half()), dict(alibi_slopes=s.cpu()),
                dict(softcap=5.0, out=torch.empty(2, 8, 64, device=DEV)),
                dict(softcap=5.0, q=q.float()), dict(softcap=5.0, q=q.transpose(0, 1)), dict(softcap=5.0, ctx=ctx[:1]),
                dict(softcap=5.0, ctx=ctx.long()), dict(softcap=5.0, err=torch.zeros(1, device=DEV))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=5.0, path=3),
                dict(softcap=5.0, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pk.PkvdError):
            call(**bad)
    for bad in (dict(prefix_lens=ctx[:1]), dict(prefix_lens=ctx.long()), dict(softcap=5.0, ck=cu[:2])):
        with pytest.raises(ValueError):
            pre(**bad)
    with pytest.raises(pk.PkvdError):
        pre(softcap=-2.0)


def test_replayed_from_a_graph_and_on_another_stream():
    pk = require_gpu()
    ctx0 = [40, 300]
    kc, vc, tables, _ = cache_of([320, 320], 8, 128, 16, torch.bfloat16, 9)
    q = torch.randn(2, 48, 128, generator=torch.Generator().manual_seed(10)).to(torch.bfloat16).to(DEV)
    s, _ = slopes_for(48, "geometric")
    ctx = torch.tensor(ctx0, dtype=torch.int32, device=DEV)
    ws = torch.empty(pk.decode_workspace_bytes(2, 48, 128, 320), dtype=torch.uint8, device=DEV)
    run = lambda **kw: pk.paged_decode_attention(q, kc, vc, tables, ctx, 320, 0.1, softcap=20.0, alibi_slopes=s, **kw)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out=out, workspace=ws)
    g.replay()
    assert torch.equal(out, want)
    ctx += 13
    q.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run())


@pytest.mark.parametrize("path", [1, 2, 3])
@pytest.mark.parametrize("prefix", [1, 128, 129, 500, 1200, 1301])
def test_prefill_prefix_far_before_the_window(prefix, path):
    """Blocks between the prefix and the window (none, one, whole tiles of them) are not read: they hold NaN, or
    are no longer in the table."""
    pk = require_gpu()
    hq, hkv, d, bs, klen, qlen, window, scale = 4, 2, 64, 16, 1400, 90, 70, 0.125
    kc, vc, tables, rows = cache_of([klen, 300], hkv, d, bs, torch.bfloat16, 7)
    first = klen - qlen + 1 - window                     # the first key in any row's window
    for b in range(-(-prefix // bs), first // bs):
        kc[tables[0, b].item()] = float("nan")
        vc[tables[0, b].item()] = float("nan")
        if b % 2:
            tables[0, b] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.randn(qlen + 20, hq, d, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    slopes = torch.full((hq,), 0.01, device=DEV)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qlen, qlen + 20], [0, klen, klen + 300]))
    out = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, qlen, scale, window=window, path=path, softcap=9.0,
                               alibi_slopes=slopes, prefix_lens=torch.tensor([prefix, 64], dtype=torch.int32, device=DEV),
                               err=err)
    assert err.item() == 0
    got, tol = out.double().cpu().numpy(), tolerances(torch.bfloat16, path != 1)
    for t in range(qlen + 20):
        i, p, n = (0, klen - qlen + t, klen) if t < qlen else (1, 300 - 20 + t - qlen, 300)
        for h in range(0, hq, 3):
            k, v = (x[:, h // (hq // hkv)] for x in rows[i])
            want, bound = oracle.scores.attend(q[t, h].double().numpy(), k, v, p, scale, 9.0, float(slopes[h]), window,
                                               (prefix, 64)[i], **tol)
            assert np.all(np.abs(got[t, h] - want) <= bound), (t, h)


@pytest.mark.parametrize("mod", [(4.0, None, 0, False), (0.0, "geometric", 0, True), (3.0, "mixed", 100, True)],
                         ids=["cap", "bias-prefix", "all"])
@pytest.mark.parametrize("case", [("f16", 16, 16, 64, 64), ("bf16", 64, 8, 64, 16), ("bf16", 48, 8, 128, 32),
                                  ("f16", 20, 10, 128, 16)], ids=lambda c: "-".join(map(str, c)))
def test_prefill_of_more_tiles_than_sms(case, mod):
    """Batches whose Q tiles outnumber the SMs several times: pairs of tiles, CTAs that take over further items."""
    pk = require_gpu()
    dt, hq, hkv, d, bs = case
    cap, kind, window, open_prefix = mod
    dt = DT[dt]
    qlen = [300, 129, 1, 0, 200, 257, 33, 280, 64, 128]
    klen = [n + c for n, c in zip(qlen, [0, 50, 700, 9, 0, 130, 400, 300, 64, 0])]
    kc, vc, tables, rows = cache_of(klen, hkv, d, bs, dt, 11)
    q = (2 * torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(12))).to(dt)
    cq, ck = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (qlen, klen))
    dev_slopes, slopes = slopes_for(hq, kind)
    prefix = [(97 * i) % (n + 40) if open_prefix else 0 for i, n in enumerate(klen)]
    pl = torch.tensor(prefix, dtype=torch.int32, device=DEV) if open_prefix else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, max(qlen), d ** -0.5, window=window, err=err, path=3,
                               softcap=cap, alibi_slopes=dev_slopes, prefix_lens=pl)
    assert err.item() == 0
    got, tol, t0 = out.double().cpu().numpy(), tolerances(dt, True), 0
    for i, n in enumerate(klen):
        for j in sorted({0, qlen[i] - 1, *range(i, qlen[i], 23)} if qlen[i] else ()):
            for h in ((j + i) % hq, hq - 1 - j % hq):
                k, v = (x[:, h // (hq // hkv)] for x in rows[i])
                want, bound = oracle.scores.attend(q[t0 + j, h].double().numpy(), k, v, n - qlen[i] + j, d ** -0.5, cap,
                                                   slopes[h], window, min(prefix[i], n), **tol)
                assert np.all(np.abs(got[t0 + j, h] - want) <= bound), (i, j, h)
        t0 += qlen[i]


def test_calls_on_two_streams_at_once():
    """Prefill and decode calls of different shapes on two streams, launched in turn: each result as when it runs alone."""
    pk = require_gpu()
    calls = []
    for seed, (dt, hq, hkv, d, bs, mod) in enumerate([
            ("bf16", 48, 8, 128, 16, dict(softcap=5.0)), ("f16", 32, 8, 64, 64, dict(prefix=True, alibi=True)),
            ("bf16", 64, 8, 64, 16, dict(softcap=9.0, alibi=True)), ("f16", 16, 8, 128, 32, dict(alibi=True))]):
        dt = DT[dt]
        qlen, klen = [200, 150, 77, 1], [900, 150, 300, 513]
        kc, vc, tables, _ = cache_of(klen, hkv, d, bs, dt, 20 + seed)
        q = torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(seed)).to(dt).to(DEV)
        cq, ck = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (qlen, klen))
        ctx = torch.tensor(klen, dtype=torch.int32, device=DEV)
        kw = dict(softcap=mod.get("softcap", 0.0), alibi_slopes=slopes_for(hq, "geometric")[0] if mod.get("alibi") else None)
        pl = torch.tensor([64, 0, 200, 513], dtype=torch.int32, device=DEV) if mod.get("prefix") else None
        calls.append(lambda s, a=(kc, vc, tables), q=q, cq=cq, ck=ck, kw=kw, pl=pl, d=d, m=max(qlen): pk.prefill_attention(
            q, *a, cq, ck, m, d ** -0.5, stream=s, prefix_lens=pl, **kw))
        calls.append(lambda s, a=(kc, vc, tables), q=q[:4].contiguous(), ctx=ctx, kw=kw, d=d: pk.paged_decode_attention(
            q, *a, ctx, 1000, d ** -0.5, stream=s, **dict(kw, softcap=kw["softcap"] or 3.0)))
    alone = [c(None).clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(6):
        for i in range(len(calls)):
            j = (i + turn) % len(calls)
            got.append((j, calls[j](streams[(i + turn // 3) % 2])))
    torch.cuda.synchronize()
    for j, out in got:
        assert torch.equal(out, alone[j]), j


def test_blocks_past_32_bit_offsets():
    """The same rows in a small pool and at the end of one of 2^31 elements and more: stores and both attentions alike."""
    pk = require_gpu()
    hq, hkv, d, bs, dt = 16, 8, 128, 16, torch.bfloat16
    nb = 2 ** 31 // (bs * hkv * d) + 64
    kc, vc, tables, _ = cache_of([300, 77], hkv, d, bs, dt, 31)
    big = [torch.empty(nb, bs, hkv, d, dtype=dt, device=DEV) for _ in range(2)]
    for small, b in zip((kc, vc), big):
        b[nb - small.shape[0]:] = small
    far = torch.where(tables >= 0, tables + (nb - kc.shape[0]), tables)
    g = torch.Generator().manual_seed(32)
    q = torch.randn(90, hq, d, generator=g).to(dt).to(DEV)
    k, v = (torch.randn(90, hkv, d, generator=g).to(dt).to(DEV) for _ in range(2))
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 60, 90], [0, 300, 377]))
    ctx = torch.tensor([300, 77], dtype=torch.int32, device=DEV)
    inv, _ = pk.rope_inv_freq(d, device=DEV)
    s = slopes_for(hq, "geometric")[0]
    got = []
    for kk, vv, t in ((kc, vc, tables), (*big, far)):
        a = pk.rope_store_prefill(q, k, v, t, cq, ck, inv, kk, vv)
        b = pk.rope_store_paged(q[:2].contiguous(), k[:2].contiguous(), v[:2].contiguous(), t, ctx, inv, kk, vv)
        got.append([a, b, *(pk.prefill_attention(a, kk, vv, t, cq, ck, 60, 0.1, path=path, softcap=4.0, alibi_slopes=s)
                            for path in (1, 2, 3)),
                    *(pk.paged_decode_attention(b, kk, vv, t, ctx, 300, 0.1, path=path, softcap=4.0, alibi_slopes=s)
                      for path in (1, 2))])
    for small, large in zip(*got):
        assert torch.equal(small, large)
    assert torch.equal(kc[tables[0, 0].item()], big[0][far[0, 0].item()])
    assert torch.equal(vc[tables[1, 4].item()][:13], big[1][far[1, 4].item()][:13])     # the row stored last among them


@pytest.mark.parametrize("mod", [(3.0, None, 0, 0), (0.0, 2.0 ** -12, 0, 70000), (20.0, 2.0 ** -14, 90000, 500)],
                         ids=["cap", "bias", "all"])
def test_a_long_context(mod):
    """150,000 keys: the chain of K tiles, a prefix and a window of thousands of tiles, and decode over the same rows."""
    pk = require_gpu()
    cap, slope, window, prefix = mod
    n, qn, hq, d, bs, dt = 150001, 40, 2, 64, 64, torch.float16
    kc, vc, tables, rows = cache_of([n], 1, d, bs, dt, 41, spare=0)
    q = (3 * torch.randn(qn, hq, d, generator=torch.Generator().manual_seed(42))).to(dt)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    slopes = None if slope is None else torch.tensor([slope, 2 * slope], device=DEV)
    pl = torch.tensor([prefix], dtype=torch.int32, device=DEV) if prefix else None
    out = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, qn, 0.125, window=window, path=3, softcap=cap,
                               alibi_slopes=slopes, prefix_lens=pl).double().cpu().numpy()
    one = pk.paged_decode_attention(q[-1:].to(DEV), kc, vc, tables, ck[1:], n, 0.125, window=window, softcap=cap or 1e4,
                                    alibi_slopes=slopes).double().cpu().numpy()
    k, v = (x[:, 0] for x in rows[0])
    tol = tolerances(dt, True)
    for h in range(hq):
        sl = (slope or 0.0) * (h + 1)
        for t in (0, 17, qn - 1):
            want, bound = oracle.scores.attend(q[t, h].double().numpy(), k, v, n - qn + t, 0.125, cap, sl, window, prefix, **tol)
            assert np.all(np.abs(out[t, h] - want) <= bound), (h, t)
        want, bound = oracle.scores.attend(q[-1, h].double().numpy(), k, v, n - 1, 0.125, cap or 1e4, sl, window, **tolerances(dt, False))
        assert np.all(np.abs(one[0, h] - want) <= bound), h


@pytest.mark.parametrize("large", [0, 30000, 59990])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_many_small_weights_beside_a_large_one(dt, large):
    """One key e^11 above 60,000 equal ones, which together outweigh it: each of their weights is 2^-16 of the largest."""
    pk = require_gpu()
    n, d, bs, dt = 60000, 64, 256, DT[dt]
    kc, vc, tables, rows = cache_of([n], 1, d, bs, dt, 51, spare=0)
    k = torch.zeros(n, d, dtype=dt)
    k[large, 0] = 22.0
    v = (1.0 + 0.25 * torch.randn(n, 1, d, generator=torch.Generator().manual_seed(52))).to(dt)
    for b in range(-(-n // bs)):
        m = min(bs, n - b * bs)
        kc[tables[0, b].item(), :m, 0], vc[tables[0, b].item(), :m] = k[b * bs:b * bs + m].to(DEV), v[b * bs:b * bs + m].to(DEV)
    q = torch.zeros(9, 1, d, dtype=dt)
    q[:, 0, 0] = 4.0
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 9], [0, n]))
    for cap in (0.0, 100.0):
        out = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, 9, 0.125, path=3, softcap=cap,
                                   alibi_slopes=torch.zeros(1, device=DEV)).double().cpu().numpy()
        for t in (0, 8):
            want, bound = oracle.scores.attend(q[t, 0].double().numpy(), k.double().numpy(), v[:, 0].double().numpy(),
                                               n - 9 + t, 0.125, cap, **tolerances(dt, True))
            assert np.all(np.abs(out[t, 0] - want) <= bound), (cap, t, np.abs(out[t, 0] - want).max(), bound.max())
