"""Pins of the modified-score oracle, and the host checks of its entry points."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from test_abi import _cache


def test_without_modifiers_it_is_softmax_attention():
    rng = np.random.default_rng(0)
    q, K, V = rng.normal(size=8), rng.normal(size=(20, 8)), rng.normal(size=(20, 8))
    for p, w in [(19, 0), (7, 0), (19, 5), (3, 9)]:
        first = max(0, p + 1 - w) if w else 0
        want = oracle.attention.attend(q, K[first:p + 1], V[first:p + 1], 0.3)
        assert np.abs(oracle.scores.attend(q, K, V, p, 0.3, window=w)[0] - want).max() < 1e-14


def test_cap_bias_and_prefix_closed_forms():
    V = np.eye(4)
    q = np.array([1.0])
    K = np.array([[1e6], [1e6], [-1e6], [0.0]])
    # scores saturate at the cap: e^5, e^5, e^-5, 1
    out, _ = oracle.scores.attend(q, K, V, 3, 1.0, cap=5.0)
    w = np.exp([5.0, 5.0, -5.0, 0.0])
    assert np.allclose(out, w / w.sum(), atol=1e-15)
    # equal keys: the bias alone decides
    out, _ = oracle.scores.attend(q, K * 0, V, 2, 1.0, slope=0.5)
    w = np.exp([-1.0, -0.5, 0.0])
    assert np.allclose(out, np.append(w / w.sum(), 0.0))
    # a prefix opens later keys, at their distance, and outlives the window
    out, _ = oracle.scores.attend(q, K * 0, V, 1, 1.0, slope=0.5, prefix=4)
    w = np.exp([-0.5, 0.0, -0.5, -1.0])
    assert np.allclose(out, w / w.sum())
    assert list(oracle.scores.visible_keys(5, 8, window=2, prefix=1)) == [1, 0, 0, 0, 1, 1, 0, 0]
    # a large cap changes nothing
    rng = np.random.default_rng(1)
    q, K, V = rng.normal(size=8), rng.normal(size=(9, 8)), rng.normal(size=(9, 8))
    assert np.allclose(oracle.scores.attend(q, K, V, 8, 1.0, cap=1e7)[0], oracle.scores.attend(q, K, V, 8, 1.0)[0])


@pytest.mark.parametrize("slopes", [False, True])
def test_against_a_masked_softmax_of_torch(slopes):
    g = torch.Generator().manual_seed(2)
    n, c = 12, 5
    q = torch.randn(n - c, 16, generator=g, dtype=torch.float64)
    K, V = (torch.randn(n, 16, generator=g, dtype=torch.float64) for _ in range(2))
    p, j = torch.arange(c, n)[:, None], torch.arange(n)[None]
    s = 3 * torch.tanh(q @ K.T * 0.5 / 3) - (0.25 * (p - j).abs() if slopes else 0)
    s = s.masked_fill(~((j <= p) | (j < 8)), float("-inf"))
    want = (torch.softmax(s, -1) @ V).numpy()
    for i in range(n - c):
        got, _ = oracle.scores.attend(q[i].numpy(), K.numpy(), V.numpy(), c + i, 0.5, cap=3.0,
                                      slope=0.25 if slopes else 0.0, prefix=8)
        assert np.abs(got - want[i]).max() < 1e-13


def test_polynomial_of_the_capped_scores():
    """The tanh(y) / y polynomials hold the errors that the kernels count on, over all of their ranges."""
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "paged_kv_decode_store_gb300", "csrc", "score_mod.cuh")).read()
    four = [float(x) for x in re.findall(r"(-?[\d.]+(?:e-?\d+)?)f", text[text.index("PKVD_TANH_RATIO4 {"):].split("}")[0])]
    body = text[text.index("float tanh_ratio6"):].split("return")[0]
    lead, *rest = re.findall(r"fmaf\(z, (-?[\d.]+)f, (-?[\d.]+)f\)|r, (-?[\d.]+)f", body)
    six = [float(lead[0]), float(lead[1])] + [float(r[2]) for r in rest]
    six = six[::-1]
    six = [float(re.search(r"return fmaf\(z, r, ([\d.]+)f\);", text).group(1))] + six
    near = float(re.search(r"kTanhNear = ([\d.]+)f", text).group(1))
    for coef, n, end, most in ((four, 4, near, 7.25e-6), (six, 6, 1.0, 6.0e-7)):
        y = np.linspace(1e-6, end, 100001)
        z = y * y
        ratio = sum(c * z ** i for i, c in enumerate(coef))
        assert len(coef) == n
        assert np.abs(ratio * y / np.tanh(y) - 1).max() < most


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk.lib()


def _mod(cap=0.0, slopes=None, prefix=None):
    from paged_kv_decode_store_gb300._capi import PkvdScoreMod
    return PkvdScoreMod(cap, slopes, prefix)


def test_score_mod_host_checks(L):
    def decode(m, scale=0.088, hq=48, window=0, n=4, ws=1 << 20):
        return L.pkvd_paged_decode_attention_mod(1 << 21, 1 << 22, ctypes.byref(_cache()), 1 << 23, 8, 1 << 24, 128, n,
                                                 hq, scale, window, m, 1 << 25, ws, None, None, 0)
    def prefill(m, scale=0.088, window=0, n=4):
        return L.pkvd_prefill_attention_mod(1 << 21, 1 << 22, ctypes.byref(_cache()), 1 << 23, 8, 1 << 24, 1 << 25, n,
                                            100, 64, 48, scale, window, m, None, None, 0)
    for call in (decode, prefill):                       # every call is answered on the host
        assert call(_mod(-1.0)) == 1
        assert call(_mod(float("nan"))) == 1
        assert call(_mod(float("inf"))) == 1
        assert call(_mod(1e-40)) == 1                    # scale / cap overflows
        assert call(_mod(3e38)) == 1                     # cap * log2(e) overflows
        assert call(_mod(30.0), scale=float("nan")) == 1
        assert call(_mod(30.0), window=-1) == 1
        assert call(_mod(30.0, 1 << 26, 1 << 27), n=0) == 0
        assert call(None, n=0) == 0
    assert decode(_mod(30.0), hq=44) == 3
    assert decode(_mod(30.0), ws=16) in (4, 5)           # too small (5: no device to ask)
