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
from ._capi import array, check, current_stream, err_ptr, on_stream, rows3

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


def _out(out, x, shape, name):
    """(tensor, token stride, pointer) of an output like x; a fresh one is contiguous."""
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        return out, max(shape[1] * shape[2], 1), out.data_ptr()
    _, stride, p = rows3(out, name, x.dtype, x.device, shape)
    return out, stride, p


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
         interleaved: bool = False, mscale: float = 1.0, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """(q, k) rotated by positions (int64 [tokens]); inv_freq float64
    [rotary_dim / 2].  q_out / k_out may be q / k (in place); k may be None."""
    dt, dev = q.dtype, q.device
    code = _capi.dtype_code(dt)
    if not q.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    qshape, qs, qp = rows3(q, "q", dt, dev)
    T, Hq, D = qshape
    ks = kos = hk = 0
    kp = kop = None
    with on_stream(stream, dev):
        q_out, qos, qop = _out(q_out, q, qshape, "q_out")
        if k is not None:
            kshape, ks, kp = rows3(k, "k", dt, dev)
            hk = kshape[1]
            if kshape[0] != T or kshape[2] != D:
                raise ValueError("k must have q's tokens and head_dim")
            k_out, kos, kop = _out(k_out, k, kshape, "k_out")
        desc = _desc(inv_freq, interleaved, mscale, dev)
        check(_capi.lib().pkvd_rope(qop, qos, qp, qs, kop, kos, kp, ks, code, T, Hq, hk, D,
                                    array(positions, "positions", torch.int64, dev, (T,)), desc,
                                    current_stream(dev)))
    return q_out, k_out


def _store(q, k, v, k_cache, v_cache):
    """The checks of a fused store's rows: (cache, q's shape, tokens, strides and pointers)."""
    c = _capi.cache_desc(k_cache, v_cache)
    dt, dev = k_cache.dtype, k_cache.device
    qshape, qs, qp = rows3(q, "q", dt, dev)
    T = qshape[0]
    if qshape[2] != c.head_dim:
        raise ValueError("q must have the cache's head_dim")
    rows = (T, c.num_kv_heads, c.head_dim)
    _, ks, kp = rows3(k, "k", dt, dev, rows)
    _, vs, vp = rows3(v, "v", dt, dev, rows)
    return c, dev, qshape, T, (qp, qs, kp, ks, vp, vs)


def rope_store_paged(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                     context_lens: torch.Tensor, inv_freq: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                     q_out: torch.Tensor | None = None, slot_mapping: torch.Tensor | None = None,
                     err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode step: row i's q and k turned by position context_lens[i] - 1, the
    key and the value stored in that token's cache slot (kv_store_paged), the
    rotated q returned (q_out may be q; rows without a context get zeros)."""
    c, dev, qshape, B, rows = _store(q, k, v, k_cache, v_cache)
    with on_stream(stream, dev):
        q_out, qos, qop = _out(q_out, q, qshape, "q_out")
        desc = _desc(inv_freq, interleaved, mscale, dev)
        tables = array(block_tables, "block_tables", torch.int32, dev, (B, None))
        check(_capi.lib().pkvd_rope_store_paged(
            qop, qos, *rows, qshape[1], tables, block_tables.shape[1],
            array(context_lens, "context_lens", torch.int32, dev, (B,)), B, desc,
            None if slot_mapping is None else array(slot_mapping, "slot_mapping", torch.int64, dev, (B,)), c,
            current_stream(dev), err_ptr(err, dev)))
    return q_out


def rope_store_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                       cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, inv_freq: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
                       q_out: torch.Tensor | None = None, slot_mapping: torch.Tensor | None = None,
                       err: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Varlen prefill batch (kv_store_prefill's rows and positions): q and k
    turned, k and v stored, the rotated q returned.  Rows past
    cu_seqlens_q[-1] of q_out and the cache stay as they were."""
    c, dev, qshape, T, rows = _store(q, k, v, k_cache, v_cache)
    n = cu_seqlens_q.shape[0] - 1
    with on_stream(stream, dev):
        q_out, qos, qop = _out(q_out, q, qshape, "q_out")
        desc = _desc(inv_freq, interleaved, mscale, dev)
        tables = array(block_tables, "block_tables", torch.int32, dev, (n, None))
        check(_capi.lib().pkvd_rope_store_prefill(
            qop, qos, *rows, qshape[1], tables, block_tables.shape[1],
            array(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, (n + 1,)),
            array(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev, (n + 1,)), n, T, desc,
            None if slot_mapping is None else array(slot_mapping, "slot_mapping", torch.int64, dev, (T,)), c,
            current_stream(dev), err_ptr(err, dev)))
    return q_out
