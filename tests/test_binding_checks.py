"""Checks of the binding that need no GPU: they come before any pointer is taken."""
import pytest
import torch

from paged_kv_decode_store_gb300 import _capi


def test_key_and_value_caches_share_type_and_device():
    """A V cache of smaller elements has K's shape and strides, but not its bytes: a store would run past its end."""
    k = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError, match="dtype and device"):
        _capi.cache_desc(k, k.to(torch.bfloat16))
    with pytest.raises(ValueError, match="dtype and device"):
        _capi.cache_desc(k, torch.zeros(4, 16, 2, 64, device="meta"))
    with pytest.raises(ValueError, match="CUDA"):          # alike, but on the host
        _capi.cache_desc(k, k.clone())
