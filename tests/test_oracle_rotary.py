"""Pins of the rotary oracle, and the host side of the rotary entry points."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from test_abi import _cache


def _inv(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(0)
    inv = _inv(16)
    q, k = rng.normal(size=(1, 1, 24)), rng.normal(size=(1, 1, 24))
    at = lambda x, p: oracle.rotary.rotate(x, [p], inv, interleaved)[0, 0]
    assert np.array_equal(at(q, 0), q[0, 0])
    assert np.array_equal(at(q, 77)[16:], q[0, 0, 16:])
    for p, s in [(5, 3), (1002, 1000), (2 ** 40 + 2, 2 ** 40)]:
        assert abs(at(q, p) @ at(k, s) - at(q, 2) @ at(k, 0)) < 1e-9
        assert abs(np.linalg.norm(at(q, p)) - np.linalg.norm(q)) < 1e-12
    # turning back
    assert np.abs(oracle.rotary.rotate(at(q, 9)[None, None], [-9], inv, interleaved) - q).max() < 1e-12


def test_angles_of_far_positions():
    assert oracle.rotary.angle(3, 0.5) == 1.5
    assert abs(oracle.rotary.angle(10 ** 6, 1.0) - math.fmod(1e6, 2 * math.pi)) < 1e-9
    assert abs(math.sin(oracle.rotary.angle(710, 113 / 710)) - math.sin(113)) < 1e-12


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk.lib()


def _freqs(L, rot, base, scaling, factor=1.0, length=4096, fast=32.0, slow=1.0):
    out = np.zeros(max(rot // 2, 1) if rot > 0 else 1)
    m = ctypes.c_float(0)
    st = L.pkvd_rope_inv_freq(out.ctypes.data, ctypes.byref(m), rot, base, scaling, factor, length, fast, slow)
    return st, out, m.value


def test_inverse_frequencies(L):
    for rot in (2, 32, 64, 128):
        st, plain, m = _freqs(L, rot, 10000.0, 0)
        assert st == 0 and m == 1.0 and np.allclose(plain, _inv(rot), rtol=1e-14)
        st, lin, m = _freqs(L, rot, 10000.0, 1, 8.0)
        assert st == 0 and m == 1.0 and np.allclose(lin, plain / 8, rtol=1e-14)
        st, ntk, m = _freqs(L, rot, 10000.0, 2, 8.0)
        want = _inv(rot, 10000.0 * 8.0 ** (rot / (rot - 2))) if rot > 2 else _inv(rot)
        assert st == 0 and np.allclose(ntk, want, rtol=1e-12)
        if rot > 2:                     # the slowest pair is stretched by exactly the factor
            assert abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-12
        st, parts, m = _freqs(L, rot, 10000.0, 3, 8.0)
        assert st == 0 and abs(m - (0.1 * math.log(8.0) + 1)) < 1e-6
        assert np.all(parts <= plain * (1 + 1e-12)) and np.all(parts >= plain / 8 * (1 - 1e-12))
    # by parts, 64 dims: fast pairs kept, slow ones divided, a ramp between
    st, plain, _ = _freqs(L, 64, 10000.0, 0)
    st, parts, _ = _freqs(L, 64, 10000.0, 3, 8.0, 4096)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(parts[turns > 48], plain[turns > 48]) and np.allclose(parts[turns < 0.7], plain[turns < 0.7] / 8)
    assert np.all(np.diff(parts / plain) <= 1e-15)


def test_inverse_frequency_refusals(L):
    assert _freqs(L, 0, 1e4, 0)[0] == 1
    assert _freqs(L, 33, 1e4, 0)[0] == 1
    assert _freqs(L, 514, 1e4, 0)[0] == 1
    assert _freqs(L, 64, 1.0, 0)[0] == 1
    assert _freqs(L, 64, float("nan"), 0)[0] == 1
    assert _freqs(L, 64, 1e4, 4)[0] == 1
    assert _freqs(L, 64, 1e4, 1, 0.5)[0] == 1
    assert _freqs(L, 64, 1e4, 3, 8.0, 0)[0] == 1
    assert _freqs(L, 64, 1e4, 3, 8.0, 4096, 1.0, 32.0)[0] == 1
    assert _freqs(L, 64, 1e4, 0, float("nan"))[0] == 0      # a plain call names no factor


P = [1 << (20 + i) for i in range(10)]                       # fake, aligned, never dereferenced


def _desc(rot=64, inter=0, m=1.0, inv=P[0]):
    from paged_kv_decode_store_gb300._capi import PkvdRope
    return ctypes.byref(PkvdRope(inv, rot, inter, m))


def test_rope_host_checks(L):
    def rope(dt=2, T=4, hq=4, hk=2, D=128, q=P[1], qs=512, qo=P[2], qos=512, k=P[3], ks=256, ko=P[4], kos=256,
             pos=P[5], desc=None):
        return L.pkvd_rope(qo, qos, q, qs, ko, kos, k, ks, dt, T, hq, hk, D, pos, desc or _desc(), None)
    # every call below is answered on the host
    assert rope(dt=3) == 2
    assert rope(T=-1) == 1
    assert rope(T=0) == 0
    assert rope(hq=0, hk=0) == 0
    assert rope(hq=-1) == 1
    assert rope(D=516) == 3
    assert rope(D=100) == 3                                  # 200 bytes: no whole 16-byte vectors
    assert rope(desc=_desc(rot=130)) == 1
    assert rope(desc=_desc(rot=0)) == 1
    assert rope(desc=_desc(rot=63)) == 3
    assert rope(desc=_desc(inter=2)) == 1
    assert rope(desc=_desc(m=float("inf"))) == 1
    assert rope(desc=_desc(inv=None)) == 1
    assert rope(desc=_desc(inv=P[0] + 4)) == 3
    assert rope(pos=None) == 1
    assert rope(pos=P[5] + 4) == 3
    assert rope(q=None) == 1
    assert rope(q=P[1] + 8) == 3
    assert rope(qs=511) == 1                                 # shorter than a row
    assert rope(qs=516) == 3                                 # 1032 bytes
    assert rope(ko=None) == 1
    assert rope(kos=248) == 1


def test_rope_store_host_checks(L):
    def paged(n=4, cache=None, desc=None, tab=P[5], ctx=P[6], q=P[1], k=P[3], vs=1024, hq=48, mb=8):
        return L.pkvd_rope_store_paged(P[2], 48 * 128, q, 48 * 128, k, 1024, P[4], vs, hq, tab, mb, ctx, n,
                                       desc or _desc(128), None, ctypes.byref(cache or _cache()), None, None)
    assert paged(n=-1) == 1
    assert paged(n=0) == 0
    assert paged(cache=_cache(head_dim=96)) == 3
    assert paged(cache=_cache(dtype=9)) == 2
    assert paged(desc=_desc(130)) == 1
    assert paged(tab=None) == 1
    assert paged(ctx=None) == 1
    assert paged(mb=0) == 1
    assert paged(q=None) == 1
    assert paged(k=P[3] + 8) == 3
    assert paged(vs=1000) == 1
    def prefill(n=4, T=9, tab=P[5], cq=P[6], ck=P[7], q=P[1], desc=None):
        return L.pkvd_rope_store_prefill(P[2], 48 * 128, q, 48 * 128, P[3], 1024, P[4], 1024, 48, tab, 8, cq, ck, n, T,
                                         desc or _desc(128), None, ctypes.byref(_cache()), None, None)
    assert prefill(n=-1) == 1
    assert prefill(T=-1) == 1
    assert prefill(T=0) == 0
    assert prefill(tab=None) == 1
    assert prefill(cq=None) == 1
    assert prefill(ck=None) == 1
    assert prefill(q=P[1] + 2) == 3
    assert prefill(desc=_desc(-2)) == 1


def test_rows_turned_in_place_keep_their_stride(L):
    def rope(q=P[1], qs=512, qo=P[2], qos=512, k=P[3], ks=256, ko=P[4], kos=256, T=4):
        return L.pkvd_rope(qo, qos, q, qs, ko, kos, k, ks, 2, T, 4, 2, 128, P[5], _desc(), None)
    assert rope(qo=P[1], qos=520) == 1
    assert rope(ko=P[3], kos=264) == 1
    def paged(qos, n):
        return L.pkvd_rope_store_paged(P[1], qos, P[1], 48 * 128, P[3], 1024, P[4], 1024, 48, P[5], 8, P[6], n,
                                       _desc(128), None, ctypes.byref(_cache()), None, None)
    assert paged(48 * 128 + 8, 2) == 1
    def prefill(qos, T):
        return L.pkvd_rope_store_prefill(P[1], qos, P[1], 48 * 128, P[3], 1024, P[4], 1024, 48, P[5], 8, P[6], P[7], 2, T,
                                         _desc(128), None, ctypes.byref(_cache()), None, None)
    assert prefill(48 * 128 + 8, 9) == 1
