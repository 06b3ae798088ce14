"""Rotary positions (include/pkvd.h, pkvd_rope*): argument marshalling only.

A row is one token's [heads, dim] with its heads side by side; the rows of q,
k and v may be slices of one projected [tokens, q + k + v heads, dim] tensor.
Every call works on the tensors' device and on ``stream`` (default: that
device's current one); what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _capi
from ._capi import array, check, current_stream, err_ptr, on_stream, ptr, rows3

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inverse frequencies, float64 [rotary_dim / 2] on `device`; factor for
    cos and sin) of a head's rotated part, scaled for contexts `factor` times
    the trained length: "none", "linear" (positions divided), "ntk" (a larger
    base) or "parts" (low frequencies divided, high ones kept, a ramp between)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    out = torch.empty(max(rotary_dim // 2, 1), dtype=torch.float64)
    m = ctypes.c_float(1.0)
    check(_capi.lib().pkvd_rope_inv_freq(out.data_ptr(), ctypes.byref(m), rotary_dim, base, _SCALINGS[scaling], factor,
                                         original_len, beta_fast, beta_slow))
    return out.to(device), float(m.value)


def _desc(inv_freq: torch.Tensor, interleaved: bool, mscale: float, device: torch.device):
    p = array(inv_freq, "inv_freq", torch.float64, device, (None,))
    return _capi.PkvdRope(p, 2 * inv_freq.shape[0], 1 if interleaved else 0, mscale)


def _out_rows(out, x, name):
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.shape != x.shape:
        raise ValueError(f"{name} must have its input's shape")
    return out


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
         interleaved: bool = False, mscale: float = 1.0, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """(q, k) rotated by positions (int64 [tokens]); inv_freq float64
    [rotary_dim / 2].  q_out / k_out may be q / k (in place); k may be None."""
    dev = q.device
    qs = rows3(q, "q")
    T, Hq, D = q.shape
    ks = kos = hk = 0
    with on_stream(stream, dev):
        q_out = _out_rows(q_out, q, "q_out")
        qos = rows3(q_out, "q_out", q)
        if k is not None:
            ks = rows3(k, "k", q)
            if k.shape[0] != T or k.shape[2] != D:
                raise ValueError("k must have q's tokens and head_dim")
            hk = k.shape[1]
            k_out = _out_rows(k_out, k, "k_out")
            kos = rows3(k_out, "k_out", q)
        desc = _desc(inv_freq, interleaved, mscale, dev)
        check(_capi.lib().pkvd_rope(ptr(q_out), qos, ptr(q), qs, ptr(k_out), kos, ptr(k), ks,
                                    _capi.dtype_code(q.dtype), T, Hq, hk, D,
                                    array(positions, "positions", torch.int64, dev, (T,)), desc,
                                    current_stream(dev)))
    return q_out, k_out


def _store_rows(q, k, v, q_out, k_cache):
    qs, ks, vs = rows3(q, "q"), rows3(k, "k", q), rows3(v, "v", q)
    _, _, Hkv, D = k_cache.shape
    T = q.shape[0]
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D) or q.shape[2] != D:
        raise ValueError("k and v must be [tokens, kv heads, head_dim] rows of the cache, q of the same head_dim")
    if k_cache.dtype != q.dtype or k_cache.device != q.device:
        raise ValueError("the cache must have the dtype and device of the rows")
    q_out = _out_rows(q_out, q, "q_out")
    return q_out, rows3(q_out, "q_out", q), qs, ks, vs


def rope_store_paged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                     context_lens: torch.Tensor, inv_freq: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                     q_out: torch.Tensor | None = None, slot_mapping: torch.Tensor | None = None,
                     err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode step: row i's q and k turned by position context_lens[i] - 1, the
    key and the value stored in that token's cache slot (kv_store_paged), the
    rotated q returned (q_out may be q; rows without a context get zeros)."""
    dev, B = q.device, q.shape[0]
    c = _capi.cache_desc(k_cache, v_cache)
    with on_stream(stream, dev):
        q_out, qos, qs, ks, vs = _store_rows(q, k, v, q_out, k_cache)
        desc = _desc(inv_freq, interleaved, mscale, dev)
        check(_capi.lib().pkvd_rope_store_paged(
            ptr(q_out), qos, ptr(q), qs, ptr(k), ks, ptr(v), vs, q.shape[1],
            array(block_tables, "block_tables", torch.int32, dev, (B, None)), block_tables.shape[1],
            array(context_lens, "context_lens", torch.int32, dev, (B,)), B, desc,
            None if slot_mapping is None else array(slot_mapping, "slot_mapping", torch.int64, dev, (B,)),
            c, current_stream(dev), err_ptr(err, dev)))
    return q_out


def rope_store_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, inv_freq: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                       q_out: torch.Tensor | None = None, slot_mapping: torch.Tensor | None = None,
                       err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Varlen prefill batch (kv_store_prefill's rows and positions): q and k
    turned, k and v stored, the rotated q returned.  Rows past
    cu_seqlens_q[-1] of q_out and the cache stay as they were."""
    dev, T = q.device, q.shape[0]
    n = cu_seqlens_q.shape[0] - 1
    c = _capi.cache_desc(k_cache, v_cache)
    with on_stream(stream, dev):
        q_out, qos, qs, ks, vs = _store_rows(q, k, v, q_out, k_cache)
        desc = _desc(inv_freq, interleaved, mscale, dev)
        check(_capi.lib().pkvd_rope_store_prefill(
            ptr(q_out), qos, ptr(q), qs, ptr(k), ks, ptr(v), vs, q.shape[1],
            array(block_tables, "block_tables", torch.int32, dev, (n, None)), block_tables.shape[1],
            array(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, (n + 1,)),
            array(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev, (n + 1,)), n, T, desc,
            None if slot_mapping is None else array(slot_mapping, "slot_mapping", torch.int64, dev, (T,)),
            c, current_stream(dev), err_ptr(err, dev)))
    return q_out
