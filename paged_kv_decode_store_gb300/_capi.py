"""ctypes declarations of include/pkvd.h and tensor-to-argument helpers."""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpkvd.so")

PATH_AUTO, PATH_FMA, PATH_MMA, PATH_TC = 0, 1, 2, 3
ERR_BLOCK_ID, ERR_SLOT, ERR_CONTEXT, ERR_TIMEOUT, ERR_TREE = 1, 2, 4, 8, 16
NO_SPACE = 6
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

c_void_p, c_int32, c_int64, c_size_t, c_float, c_double = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                           ctypes.c_size_t, ctypes.c_float, ctypes.c_double)


class PkvdCache(ctypes.Structure):
    _fields_ = [("k_base", c_void_p), ("v_base", c_void_p), ("dtype", c_int32),
                ("block_size", c_int32), ("num_blocks", c_int64), ("num_kv_heads", c_int32),
                ("head_dim", c_int32), ("block_stride", c_int64), ("token_stride", c_int64),
                ("head_stride", c_int64)]


class PkvdRope(ctypes.Structure):
    _fields_ = [("inv_freq", c_void_p), ("rotary_dim", c_int32), ("interleaved", c_int32), ("mscale", c_float)]


class PkvdScoreMod(ctypes.Structure):
    _fields_ = [("softcap", c_float), ("alibi_slopes", c_void_p), ("prefix_lens", c_void_p)]


class PkvdError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"pkvd status {status}: {text}")
        self.status = status


# name -> (restype, argtypes)
SIGNATURES = {
    "pkvd_status_string": (ctypes.c_char_p, [c_int32]),
    "pkvd_version": (c_int32, []),
    "pkvd_slot_mapping": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_int32, c_int64,
                                    c_void_p, c_void_p]),
    "pkvd_kv_store": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, ctypes.POINTER(PkvdCache),
                                c_void_p, c_void_p]),
    "pkvd_kv_store_paged": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p,
                                      ctypes.POINTER(PkvdCache), c_void_p, c_void_p]),
    "pkvd_kv_store_prefill": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                        c_int32, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_void_p]),
    "pkvd_rope": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int32,
                            c_int32, c_int32, c_int32, c_int32, c_void_p, ctypes.POINTER(PkvdRope), c_void_p]),
    "pkvd_rope_store_paged": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                        c_int32, c_void_p, c_int32, c_void_p, c_int32, ctypes.POINTER(PkvdRope),
                                        c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_void_p]),
    "pkvd_rope_store_prefill": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64,
                                          c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                          ctypes.POINTER(PkvdRope), c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                          c_void_p]),
    "pkvd_rope_inv_freq": (c_int32, [c_void_p, c_void_p, c_int32, c_double, c_int32, c_double, c_int64, c_double,
                                     c_double]),
    "pkvd_prefill_attention": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32,
                                         c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_float,
                                         c_int32, c_void_p, c_void_p]),
    "pkvd_prefill_attention_ex": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32,
                                            c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_float,
                                            c_int32, c_void_p, c_void_p, c_int32]),
    "pkvd_prefill_attention_mod": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32,
                                             c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_float,
                                             c_int32, ctypes.POINTER(PkvdScoreMod), c_void_p, c_void_p, c_int32]),
    "pkvd_beam_workspace_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, ctypes.POINTER(c_size_t)]),
    "pkvd_beam_search_step": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32,
                                        c_int64, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_size_t, c_void_p]),
    "pkvd_bm_create": (c_int32, [c_int32, c_int32, ctypes.POINTER(c_void_p)]),
    "pkvd_bm_destroy": (None, [c_void_p]),
    "pkvd_bm_num_free": (c_int32, [c_void_p]),
    "pkvd_bm_ref_count": (c_int32, [c_void_p, c_int32]),
    "pkvd_bm_allocate": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, ctypes.POINTER(c_int32),
                                   ctypes.POINTER(c_int32)]),
    "pkvd_bm_append": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, ctypes.POINTER(c_int32), c_int32,
                                 ctypes.POINTER(c_int32), ctypes.POINTER(c_int32), ctypes.POINTER(c_int32)]),
    "pkvd_bm_fork": (c_int32, [c_void_p, c_void_p, c_int32]),
    "pkvd_bm_reorder": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "pkvd_bm_shared_prefix": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_int32, ctypes.POINTER(c_int32)]),
    "pkvd_bm_release": (c_int32, [c_void_p, c_void_p, c_int32]),
    "pkvd_copy_blocks": (c_int32, [ctypes.POINTER(PkvdCache), c_void_p, c_void_p, c_void_p, c_int32, c_void_p,
                                   c_void_p]),
    "pkvd_decode_workspace_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32,
                                              ctypes.POINTER(c_size_t)]),
    "pkvd_paged_decode_attention": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                              c_int32, c_void_p, c_int32, c_int32, c_int32, c_float,
                                              c_void_p, c_size_t, c_void_p, c_void_p]),
    "pkvd_paged_decode_attention_ex": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                                 c_int32, c_void_p, c_int32, c_int32, c_int32, c_float,
                                                 c_void_p, c_size_t, c_void_p, c_void_p, c_int32]),
    "pkvd_paged_decode_attention_window": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                                     c_int32, c_void_p, c_int32, c_int32, c_int32, c_float,
                                                     c_int32, c_void_p, c_size_t, c_void_p, c_void_p, c_int32]),
    "pkvd_paged_decode_attention_mod": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                                  c_int32, c_void_p, c_int32, c_int32, c_int32, c_float,
                                                  c_int32, ctypes.POINTER(PkvdScoreMod), c_void_p, c_size_t,
                                                  c_void_p, c_void_p, c_int32]),
    "pkvd_decode_prefix_workspace_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32,
                                                     ctypes.POINTER(c_size_t)]),
    "pkvd_paged_decode_attention_prefix": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32,
                                                     c_void_p, c_int32, c_int32, c_int32, c_float, c_int32, c_void_p,
                                                     c_size_t, c_void_p, c_void_p]),
    "pkvd_paged_decode_attention_noalloc": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p,
                                                      c_int32, c_void_p, c_int32, c_int32, c_int32, c_float,
                                                      c_void_p, c_void_p]),
    "pkvd_tree_workspace_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_int32,
                                            ctypes.POINTER(c_size_t)]),
    "pkvd_tree_attention": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32, c_void_p,
                                      c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_float, c_int32,
                                      ctypes.POINTER(PkvdScoreMod), c_void_p, c_size_t, c_void_p, c_void_p, c_int32]),
    "pkvd_tree_accept": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p]),
    "pkvd_compact_cache": (c_int32, [ctypes.POINTER(PkvdCache), c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_int64,
                                     c_int64, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "pkvd_decode_weights_workspace_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32,
                                                      ctypes.POINTER(c_size_t)]),
    "pkvd_paged_decode_attention_weights": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(PkvdCache), c_void_p, c_int32,
                                                      c_void_p, c_int32, c_int32, c_int32, c_float, c_int32,
                                                      ctypes.POINTER(PkvdScoreMod), c_void_p, c_void_p, c_int64,
                                                      c_int64, c_int32, c_void_p, c_size_t, c_void_p, c_void_p,
                                                      c_int32]),
    "pkvd_evict_select": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int32, c_void_p,
                                    c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p]),
    "pkvd_bm_reserve": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, ctypes.POINTER(c_int32), c_int32,
                                  ctypes.POINTER(c_int32), ctypes.POINTER(c_int32), ctypes.POINTER(c_int32)]),
    "pkvd_bm_trim": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, ctypes.POINTER(c_int32)]),
    "pkvd_bm_evict": (c_int32, [c_void_p, c_int32, c_void_p, ctypes.POINTER(c_int32)]),
    "pkvd_sample_workspace_bytes": (c_int32, [c_int32, c_int32, ctypes.POINTER(c_size_t)]),
    "pkvd_sample": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_void_p,
                              c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "pkvd_sample_ex": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int64, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_size_t, c_void_p]),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def check(status: int) -> None:
    if status != 0:
        raise PkvdError(status, lib().pkvd_status_string(status).decode())


def dtype_code(dt: torch.dtype) -> int:
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    return _DTYPES[dt]


def ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on a CUDA device")
    return t.data_ptr()


def stream_handle(stream, like: torch.Tensor):
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


_HERE = contextlib.nullcontext()
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def on_stream(stream, device: torch.device):
    """Context in which `device` is current and allocations and launches go to
    `stream` (a torch stream or a raw handle; None: the device's current one),
    so what a call allocates belongs to the stream that uses it."""
    if stream is None:
        return _HERE if device.index == _current_device() else torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


def current_stream(device: torch.device) -> int:
    """Handle of the device's current stream (torch's own short way to it where there is one)."""
    return _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def rows3(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, shape: tuple | None = None):
    """Check [tokens, heads, dim] rows whose heads lie side by side (a token's
    row may be a slice of a longer one): (shape, token stride in elements,
    pointer)."""
    have = t.shape
    if len(have) != 3 or t.dtype is not dtype or t.device != device or (shape is not None and have != shape):
        raise ValueError(f"{name} must be a {dtype} tensor [tokens, heads, dim] on {device}"
                         + (f" of shape {list(shape)}" if shape is not None else ""))
    T, H, D = have
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return have, (st if T > 1 else max(H * D, 1)), t.data_ptr()


def array(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, shape: tuple) -> int:
    """Check a contiguous argument array (None as the last size: any) and give its pointer."""
    have = t.shape
    if t.dtype is not dtype or t.device != device or not t.is_contiguous() or \
            (have != shape and (len(have) != len(shape) or shape[-1] is not None or have[:-1] != shape[:-1])):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"{[('any' if n is None else n) for n in shape]} on {device}")
    return t.data_ptr()


def err_ptr(err, device: torch.device):
    """The optional error flag: one int32 on the call's device."""
    if err is None:
        return None
    if err.dtype != torch.int32 or err.device != device or err.numel() < 1:
        raise ValueError(f"err must be an int32 tensor on {device}")
    return err.data_ptr()


def score_mod(softcap: float, alibi_slopes, prefix_lens, num_q_heads: int, num_seqs: int, device: torch.device):
    """The pkvd_score_mod of an attention call, or None when nothing is on."""
    if not softcap and alibi_slopes is None and prefix_lens is None:
        return None
    slopes = None if alibi_slopes is None else array(alibi_slopes, "alibi_slopes", torch.float32, device,
                                                     (num_q_heads,))
    prefix = None if prefix_lens is None else array(prefix_lens, "prefix_lens", torch.int32, device, (num_seqs,))
    return PkvdScoreMod(softcap, slopes, prefix)


def rows_like(q, out, k_cache):
    """q and out of an attention call: contiguous rows of the cache's type and head_dim."""
    if q.dim() != 3 or not q.is_contiguous() or q.dtype != k_cache.dtype or q.device != k_cache.device or \
            q.shape[2] != k_cache.shape[3]:
        raise ValueError("q must be contiguous [rows, heads, head_dim] of the cache's dtype and device")
    if out is None:
        return torch.empty_like(q)
    if out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor like q")
    return out


def scratch(workspace, nbytes: int, device: torch.device):
    """A call's workspace: the caller's, or one of its own."""
    if workspace is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def cache_desc(k_cache: torch.Tensor, v_cache: torch.Tensor) -> PkvdCache:
    """Describe [num_blocks, block_size, Hkv, D] views (e.g. kv_cache[0, layer])."""
    shape, stride = k_cache.shape, k_cache.stride()
    if shape != v_cache.shape or stride != v_cache.stride():
        raise ValueError("K and V caches must share shape and strides")
    if k_cache.dtype is not v_cache.dtype or k_cache.device != v_cache.device:
        raise ValueError("K and V caches must share dtype and device")
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError("cache views must be [num_blocks, block_size, Hkv, D] with D contiguous")
    nb, bs, H, D = shape
    return PkvdCache(ptr(k_cache), ptr(v_cache), dtype_code(k_cache.dtype), bs, nb, H, D, stride[0], stride[1],
                     stride[2])
