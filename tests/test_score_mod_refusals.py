"""Refusals of the attention calls with score modifiers that come before any work (no GPU)."""
import ctypes

import pytest

from paged_kv_decode_store_gb300 import _capi

OK, INVALID_ARG = 0, 1
SOME = 1 << 20          # an aligned address that is never read: the batch is empty


def decode(window, mod, max_context=100):
    cache = _capi.PkvdCache(SOME, SOME, 2, 16, 4, 8, 64, 16 * 8 * 64, 8 * 64, 64)
    return _capi.lib().pkvd_paged_decode_attention_mod(SOME, SOME, ctypes.byref(cache), SOME, 8, SOME, max_context, 0, 8,
                                                       0.125, window, ctypes.byref(mod), None, 0, None, None, 0)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_decode_with_a_prefix_that_a_window_cuts_off(softcap):
    """Prefill keeps the prefix visible past the window; the same token by decode would lose it."""
    prefix, none = _capi.PkvdScoreMod(softcap, None, SOME), _capi.PkvdScoreMod(softcap, None, None)
    assert decode(40, prefix) == INVALID_ARG and decode(99, prefix) == INVALID_ARG
    assert decode(0, prefix) == OK and decode(100, prefix) == OK and decode(200, prefix) == OK
    assert decode(40, none) == OK


@pytest.mark.parametrize("softcap,status", [(-1.0, INVALID_ARG), (float("nan"), INVALID_ARG), (float("inf"), INVALID_ARG),
                                            (1e-40, INVALID_ARG), (3e38, INVALID_ARG), (1e-30, OK), (1e38, OK)])
def test_caps(softcap, status):
    assert decode(0, _capi.PkvdScoreMod(softcap, None, None)) == status
