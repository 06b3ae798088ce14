"""Eviction by accumulated attention weight, and the moves of cached rows
(include/pkvd.h, pkvd_paged_decode_attention_weights, pkvd_evict_select,
pkvd_compact_cache): argument marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi
from ._capi import PATH_AUTO, array, cache_desc, check, current_stream, err_ptr, on_stream, rows_like, score_mod, scratch


def decode_weights_workspace_bytes(num_seqs: int, num_q_heads: int, head_dim: int, max_context_len: int) -> int:
    """Workspace of a paged_decode_attention_weights call on the current device."""
    return _workspace_bytes(num_seqs, num_q_heads, head_dim, max_context_len, torch.cuda.current_device())


@functools.lru_cache(maxsize=256)
def _workspace_bytes(num_seqs, num_q_heads, head_dim, max_context_len, device):
    n = ctypes.c_size_t(0)
    check(_capi.lib().pkvd_decode_weights_workspace_bytes(num_seqs, num_q_heads, head_dim, max_context_len, 0,
                                                          ctypes.byref(n)))
    return int(n.value)


def _weight_rows(t: torch.Tensor, name: str, device: torch.device, rows: int):
    """(heads, length, sequence stride, head stride, pointer) of float32 [rows, heads, length]."""
    if t.dim() != 3 or t.dtype != torch.float32 or t.device != device or t.shape[0] != rows or \
            (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name} must be a float32 tensor [{rows}, heads, length] on {device}, lengths contiguous")
    return t.shape[1], t.shape[2], t.stride(0), t.stride(1), t.data_ptr()


def _weights_out(weights, weights_out):
    if weights_out.shape != weights.shape or weights_out.stride() != weights.stride() or \
            weights_out.dtype != weights.dtype or weights_out.device != weights.device:
        raise ValueError("weights_out must be a tensor like weights, at the same strides")
    return weights_out.data_ptr()


def paged_decode_attention_weights(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                                   scale: float, weights: torch.Tensor, weights_out: torch.Tensor | None = None,
                                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                   err: torch.Tensor | None = None, stream=None, path: int = PATH_AUTO, window: int = 0,
                                   softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None):
    """paged_decode_attention that also counts what each cached position was given:
    (out, weights_out) with weights_out[i, h, j] = weights[i, h, j] + the softmax
    weights of position j summed over KV head h's query heads (all of them when
    weights has one head).  weights: float32 [B, Hkv or 1, >= max_context_len], no
    two rows over one another; weights_out: a tensor like it, by default weights
    itself.  Only decoded tokens count: prefill_attention and tree_attention hand no
    weights on, so right after a prompt all are equal."""
    B, Hq, D = q.shape if q.dim() == 3 else (0, 0, 0)
    dev = q.device
    c = cache_desc(k_cache, v_cache)
    heads, length, s_seq, s_head, w = _weight_rows(weights, "weights", dev, B)
    if length < max_context_len:
        raise ValueError("weights has fewer positions than max_context_len")
    if weights_out is None:
        weights_out = weights
    with on_stream(stream, dev):
        out = rows_like(q, out, k_cache)
        m = score_mod(softcap, alibi_slopes, None, Hq, B, dev)
        nbytes = 0 if workspace is not None else _workspace_bytes(B, Hq, D, max_context_len, dev.index)
        workspace = scratch(workspace, nbytes, dev)
        check(_capi.lib().pkvd_paged_decode_attention_weights(
            out.data_ptr(), q.data_ptr(), c, array(block_tables, "block_tables", torch.int32, dev, (B, None)),
            block_tables.shape[1], array(context_lens, "context_lens", torch.int32, dev, (B,)), max_context_len, B, Hq,
            scale, window, m, _weights_out(weights, weights_out), w, s_seq, s_head, heads, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), current_stream(dev), err_ptr(err, dev), path))
    return out, weights_out


def evict_select(weights: torch.Tensor, context_lens: torch.Tensor, keep: int, sink: int = 0, recent: int = 0,
                 weights_out: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None):
    """(positions [B, heads, keep], counts [B]): the cached positions that stay when
    a sequence is cut to `keep` rows -- its first `sink`, its last `recent` and the
    heaviest of the others (float32 weights [B, heads, length]), ascending, -1
    behind.  weights_out (a tensor like weights; weights itself: in place) gets
    the weights that stay, closed up, zeros behind.  Pass positions and counts to
    compact_cache; counts are the new context_lens.

    They count rows then, not tokens, and with a list for each head a row is another
    token in each: give rope the tokens' own positions and store with kv_store_paged
    (rope_store_paged turns by context_lens - 1), and decode without window and
    alibi_slopes, which would count rows."""
    dev, B = weights.device, context_lens.shape[0]
    heads, length, s_seq, s_head, w = _weight_rows(weights, "weights", dev, B)
    with on_stream(stream, dev):
        positions = torch.empty(B, heads, max(keep, 0), dtype=torch.int32, device=dev)
        counts = torch.empty(B, dtype=torch.int32, device=dev)
        check(_capi.lib().pkvd_evict_select(
            positions.data_ptr(), counts.data_ptr(), None if weights_out is None else _weights_out(weights, weights_out),
            w, s_seq, s_head, length, array(context_lens, "context_lens", torch.int32, dev, (B,)), B, heads, keep, sink,
            recent, current_stream(dev), err_ptr(err, dev)))
    return positions, counts


def compact_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, positions: torch.Tensor,
                  counts: torch.Tensor, first: torch.Tensor | None = None, new_tables: torch.Tensor | None = None,
                  err: torch.Tensor | None = None, stream=None) -> None:
    """Rows of the cache close up: for r < counts[i], row first[i] + r (first: int32
    [S], default 0) of sequence i becomes its row positions[i, r], K and V.
    positions: int32 [S, n] or [S, 1, n] for all KV heads alike, [S, Hkv, n] for
    each its own.  In place by default (every position at least first + r, as
    ascending ones are); with new_tables the rows go to those blocks, none of
    which may be read."""
    dev, S = k_cache.device, block_tables.shape[0]
    c = cache_desc(k_cache, v_cache)
    hkv = k_cache.shape[2]
    if positions.dim() == 2:
        positions = positions.unsqueeze(1)
    if positions.dim() != 3 or positions.shape[0] != S or positions.shape[1] not in (1, hkv) or \
            positions.dtype != torch.int32 or positions.device != dev or \
            (positions.stride(2) != 1 and positions.shape[2] > 1):
        raise ValueError(f"positions must be int32 [{S}, n] or [{S}, 1 or {hkv}, n] on {dev}, n contiguous")
    with on_stream(stream, dev):
        tables = array(block_tables, "block_tables", torch.int32, dev, (S, None))
        to, width = tables, block_tables.shape[1]
        if new_tables is not None:
            to, width = array(new_tables, "new_tables", torch.int32, dev, (S, None)), new_tables.shape[1]
        check(_capi.lib().pkvd_compact_cache(
            c, tables, block_tables.shape[1], to, width, positions.data_ptr(), positions.stride(0),
            positions.stride(1) if positions.shape[1] > 1 else 0, array(counts, "counts", torch.int32, dev, (S,)),
            None if first is None else array(first, "first", torch.int32, dev, (S,)), S, positions.shape[2],
            current_stream(dev), err_ptr(err, dev)))
