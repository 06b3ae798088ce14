"""Softmax scales of zero and below, which every finite scale includes: prefill and decode, plain and with modifiers."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_score_mod import DEV, DT, cache_of, slopes_for, tolerances

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mod", [(0.0, None, 0), (0.0, None, 25), (5.0, None, 0), (5.0, "geometric", 25), (0.0, "geometric", 0)],
                         ids=["plain", "window", "cap", "cap-bias-window", "bias"])
@pytest.mark.parametrize("scale", [0.0, -0.125, -3.0])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128), ("f32", 64)])
def test_scales_that_are_not_positive(dt, d, scale, mod):
    pk = require_gpu()
    dt, (cap, kind, window) = DT[dt], mod
    hq, hkv, bs, qlen, klen = 16, 8, 16, [70, 1, 30], [70, 131, 200]
    kc, vc, tables, rows = cache_of(klen, hkv, d, bs, dt, 1)
    q = torch.randn(sum(qlen), hq, d, generator=torch.Generator().manual_seed(2)).to(dt)
    cq, ck = (torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV) for x in (qlen, klen))
    dev_slopes, slopes = slopes_for(hq, kind)
    last = torch.cumsum(torch.tensor(qlen), 0) - 1
    ctx = torch.tensor(klen, dtype=torch.int32, device=DEV)
    for path in (0, 1) if dt == torch.float32 else (0, 1, 2, 3):
        got = pk.prefill_attention(q.to(DEV), kc, vc, tables, cq, ck, max(qlen), scale, window=window, path=path,
                                   softcap=cap, alibi_slopes=dev_slopes).double().cpu().numpy()
        one = got[last.numpy()] if path == 3 else pk.paged_decode_attention(
            q[last].to(DEV), kc, vc, tables, ctx, max(klen), scale, window=window, path=path, softcap=cap,
            alibi_slopes=dev_slopes).double().cpu().numpy()
        tol, t = tolerances(dt, path != 1 and dt != torch.float32), 0
        for i, n in enumerate(klen):
            for j in range(qlen[i]):
                for h in range(0, hq, 5):
                    k, v = (x[:, h // (hq // hkv)] for x in rows[i])
                    want, bound = oracle.scores.attend(q[t, h].double().numpy(), k, v, n - qlen[i] + j, scale, cap,
                                                       slopes[h], window, **tol)
                    assert np.all(np.abs(got[t, h] - want) <= bound), (path, i, j, h)
                    if j == qlen[i] - 1:
                        assert np.all(np.abs(one[i, h] - want) <= bound), (path, i, h)
                t += 1
