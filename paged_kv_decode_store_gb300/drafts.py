"""Trees of drafted tokens (include/pkvd.h, pkvd_tree_*): argument marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi
from ._capi import PATH_AUTO, array, cache_desc, check, current_stream, err_ptr, on_stream, rows_like, score_mod, scratch


def tree_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seqlen_q: int) -> int:
    """Workspace of a tree_attention call on the current device."""
    return _workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seqlen_q, torch.cuda.current_device())


@functools.lru_cache(maxsize=256)
def _workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seqlen_q, device):
    n = ctypes.c_size_t(0)
    check(_capi.lib().pkvd_tree_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seqlen_q, 0,
                                                ctypes.byref(n)))
    return int(n.value)


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, parents: torch.Tensor, max_seqlen_q: int,
                   scale: float, window: int = 0, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, err: torch.Tensor | None = None, stream=None,
                   path: int = PATH_AUTO, softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of drafted rows q ([total_q, Hq, D]) over their sequence's cached
    tokens, their ancestors and themselves.  Sequence i's rows cu_seqlens_q[i] ..
    are the nodes of a tree stored behind its cached tokens (kv_store_prefill);
    parents (int32 [total_q]) holds each node's parent within the tree, an
    earlier node or -1.  Positions (of the window, of a distance bias, and of
    rope) are the cached length plus the node's depth."""
    T, Hq, D = q.shape if q.dim() == 3 else (0, 0, 0)
    dev, n = q.device, cu_seqlens_q.shape[0] - 1
    c = cache_desc(k_cache, v_cache)
    with on_stream(stream, dev):
        out = rows_like(q, out, k_cache)
        m = score_mod(softcap, alibi_slopes, None, Hq, n, dev)
        nbytes = 0
        if workspace is None and T and max_seqlen_q > 0:
            nbytes = _workspace_bytes(n, Hq, k_cache.shape[2], D, max_seqlen_q, dev.index)
        workspace = scratch(workspace, nbytes, dev)
        check(_capi.lib().pkvd_tree_attention(
            out.data_ptr(), q.data_ptr(), c, array(block_tables, "block_tables", torch.int32, dev, (n, None)),
            block_tables.shape[1], array(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, (n + 1,)),
            array(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev, (n + 1,)),
            array(parents, "parents", torch.int32, dev, (T,)), n, T, max_seqlen_q, Hq, scale, window, m,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), current_stream(dev), err_ptr(err, dev),
            path))
    return out


def tree_accept(drafted: torch.Tensor, parents: torch.Tensor, target: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, max_path: int, err: torch.Tensor | None = None, stream=None):
    """(positions [S, max_path], first [S], counts [S], tokens [S, max_path]): the
    path of drafted nodes that the target's own choices follow, from node 0 (the
    token chosen last) on.

    drafted, parents, target: int32 [total_q], a node's id, its parent and the id
    the target chooses after it.  positions are cache positions: pass them with
    counts and first to compact_cache; the sequence then holds first + counts
    tokens.  tokens are the step's new ids, the last of which is no draft."""
    dev, T, n = drafted.device, drafted.shape[0], cu_seqlens_q.shape[0] - 1
    with on_stream(stream, dev):
        width = max(max_path, 0)
        positions = torch.empty(n, width, dtype=torch.int32, device=dev)
        first = torch.empty(n, dtype=torch.int32, device=dev)
        counts = torch.empty(n, dtype=torch.int32, device=dev)
        tokens = torch.empty(n, width, dtype=torch.int32, device=dev)
        check(_capi.lib().pkvd_tree_accept(
            positions.data_ptr(), first.data_ptr(), counts.data_ptr(), tokens.data_ptr(),
            array(drafted, "drafted", torch.int32, dev, (T,)), array(parents, "parents", torch.int32, dev, (T,)),
            array(target, "target", torch.int32, dev, (T,)),
            array(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, (n + 1,)),
            array(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev, (n + 1,)), n, T, max_path, current_stream(dev),
            err_ptr(err, dev)))
    return positions, first, counts, tokens
