"""The cap's own accuracy on each path: scores near a cap of thousands, where its error decides the weights."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import require_gpu
from test_gpu_large_scores import check, place, rows_around
from test_gpu_score_mod import DEV, DT, tolerances

pytestmark = pytest.mark.gpu

# cap and scores (log2 units): tanh in its near and its far form, at both signs, and beyond the cap
CAPS = [(2000.0, 1500.0), (2000.0, -1500.0), (2000.0, 2800.0), (2000.0, -9000.0), (20000.0, 2500.0)]


def tolerance(dt, path):
    of = "f32" if dt == torch.float32 else "tcgen05" if path == 3 else "16-bit"
    return dict(tolerances(dt, path != 1), cap_error=oracle.scores.CAP_ERROR[of])


@pytest.mark.parametrize("cap,offset", CAPS)
@pytest.mark.parametrize("dt,d,path", [("f32", 64, 1), ("f32", 128, 1)] +
                         [(t, d, p) for t in ("f16", "bf16") for d in (64, 128) for p in (1, 2, 3)])
def test_prefill(dt, d, path, cap, offset):
    pk = require_gpu()
    dt, n, qn, hq, hkv, bs = DT[dt], 200, 9, 4, 2, 16
    q, k, v = rows_around(offset, n, qn, hq, hkv, d, dt, 1)
    kc, vc, table = place(k, v, bs, dt, 2)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    out = pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, 0.125, path=path, softcap=cap)
    check(out.double().cpu().numpy(), q, k, v, range(n - qn, n), cap, np.zeros(hq), 0, tolerance(dt, path))


@pytest.mark.parametrize("cap,offset", CAPS)
@pytest.mark.parametrize("dt,hkv,path", [("f32", 8, 1), ("f32", 2, 1), ("f16", 8, 1), ("f16", 8, 2), ("bf16", 16, 2),
                                         ("f16", 3, 0)])
def test_decode(dt, hkv, path, cap, offset):
    pk = require_gpu()
    dt, n, d, bs = DT[dt], 200, 64, 16
    q, k, v = rows_around(offset, n, 1, 2 * hkv, hkv, d, dt, 3)
    kc, vc, table = place(k, v, bs, dt, 4)
    out = pk.paged_decode_attention(q.to(DEV), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), n, 0.125,
                                    path=path, softcap=cap)
    check(out.double().cpu().numpy(), q, k, v, [n - 1], cap, np.zeros(2 * hkv), 0, tolerance(dt, path or 1))


@pytest.mark.parametrize("size", [2.0 ** 38, 2.0 ** -60])
@pytest.mark.parametrize("offset", [9000.0, -9000.0])
@pytest.mark.parametrize("cap", [30.0, 44.0])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_without_a_reference(d, cap, offset, size):
    """bf16 weights under a cap of at most 44 are 2^-64 to 2^64 as they come: every score at the cap, values at the ends
    of the range that leaves them."""
    pk = require_gpu()
    dt, n, qn, hq, hkv, bs = torch.bfloat16, 300, 9, 4, 2, 16
    q, k, v = rows_around(offset, n, qn, hq, hkv, d, dt, 5)
    v = v * size
    kc, vc, table = place(k, v, bs, dt, 6)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, qn], [0, n]))
    out = pk.prefill_attention(q.to(DEV), kc, vc, table, cq, ck, qn, 0.125, path=3, softcap=cap)
    check(out.double().cpu().numpy(), q, k, v, range(n - qn, n), cap, np.zeros(hq), 0, tolerance(dt, 3))
