"""Beam search selection (include/pkvd.h, pkvd_beam_search_step): argument
marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi
from ._capi import array, check, current_stream, on_stream


@functools.lru_cache(maxsize=256)
def beam_workspace_bytes(num_requests: int, num_beams: int, vocab: int, dtype: torch.dtype, keep: int) -> int:
    n = ctypes.c_size_t(0)
    check(_capi.lib().pkvd_beam_workspace_bytes(num_requests, num_beams, vocab, _capi.dtype_code(dtype), keep,
                                                ctypes.byref(n)))
    return int(n.value)


def beam_search_step(logits: torch.Tensor, scores: torch.Tensor, keep: int, finished: torch.Tensor | None = None,
                     eos_id: int = -1, out=None, workspace: torch.Tensor | None = None, stream=None):
    """(scores, parents, tokens), each [requests, keep]: the best continuations
    of every request over its beams and the vocabulary, best first.

    logits [requests * beams, vocab] (rows may be strided), scores float32
    [requests, beams]; finished (uint8 or bool, [requests, beams]) marks ended
    beams, which continue with eos_id alone at their own score.  out: three
    tensors to write (float32, int32, int32); its scores may be `scores` when
    keep equals the beams.  parents are beams within their request: pass them
    to BlockManager.reorder."""
    dev = logits.device
    if scores.dim() != 2:
        raise ValueError("scores must be [requests, beams]")
    n, b = scores.shape
    if logits.dim() != 2 or logits.shape[0] != n * b or not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor [requests * beams, vocab]")
    vocab = logits.shape[1]
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    row_stride = logits.stride(0) if n * b > 1 else vocab
    code = _capi.dtype_code(logits.dtype)
    ended = None
    if finished is not None:
        if finished.dtype == torch.bool:
            finished = finished.view(torch.uint8)
        ended = array(finished, "finished", torch.uint8, dev, (n, b))
    with on_stream(stream, dev):
        if out is None:
            shape = (n, max(keep, 0))
            tokens = torch.empty(shape, dtype=torch.int32, device=dev)
            out = torch.empty(shape, dtype=torch.float32, device=dev), torch.empty_like(tokens), tokens
            pointers = [t.data_ptr() for t in out]
        else:
            shape = (n, keep)
            pointers = [array(out[0], "out scores", torch.float32, dev, shape),
                        array(out[1], "out parents", torch.int32, dev, shape),
                        array(out[2], "out tokens", torch.int32, dev, shape)]
        if workspace is None:
            workspace = torch.empty(max(beam_workspace_bytes(n, b, vocab, logits.dtype, keep), 16),
                                    dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        check(_capi.lib().pkvd_beam_search_step(
            *pointers, logits.data_ptr(), code, n, b, vocab, row_stride,
            array(scores, "scores", torch.float32, dev, (n, b)), ended, eos_id, keep, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), current_stream(dev)))
    return tuple(out)
