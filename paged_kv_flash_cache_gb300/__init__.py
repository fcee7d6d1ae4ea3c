"""paged_kv_flash_cache_gb300 -- attention over a paged KV cache on NVIDIA GB300 (sm_103a).

A thin Python binding over the C ABI of libpkv (include/pkv.h). Every step of the
computation runs in the library's CUDA kernels; this module only checks tensor
shapes, dtypes and devices, allocates outputs / workspace with PyTorch when the
caller does not pass them, and forwards raw device pointers and the current CUDA
stream. There is no CPU fallback: if the library is missing every call raises.

Entry points (same names as the C ABI without the ``pkv_`` prefix):
  kv_cache_append, paged_attn_decode, paged_attn_decode_step, paged_attn_prefill, paged_attn_mixed,
  attn_combine, decode_workspace_size, decode_split_tokens, get_device_error;
  around the attention of a step, and of a step with drafted tokens: rope_append (norm, rotary positions,
  append), paged_attn_tree and tree_workspace_size (a tree of drafted tokens over the cache), kv_cache_compact
  (the rows that are kept move to the front). `rope.rope_frequencies`, `workloads.tree_mask` and
  `workloads.tree_depths` make their arguments on the host.
Cache tensors have shape [num_blocks, 2, num_kv_heads, block_size, head_dim]
(K at index 0, V at index 1) in float16 or bfloat16, or hold FP8 E4M3 codes
(torch.float8_e4m3fn or uint8) with a float32 `scales` tensor
[num_blocks, 2, num_kv_heads, block_size], one scale per cached row; q, k_new and
v_new then stay float16 / bfloat16 (see pkv_kv_format in include/pkv.h).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional

__all__ = [
    "PkvError", "library_path", "load_library", "kv_cache_append", "paged_attn_decode", "paged_attn_prefill",
    "attn_combine", "decode_workspace_size", "decode_split_tokens", "get_device_error", "STATUS",
    "paged_attn_decode_noalloc", "paged_attn_mixed", "selftest_wait_timeout", "paged_attn_decode_step",
    "rope_append", "paged_attn_tree", "tree_workspace_size", "kv_cache_compact",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libpkv.so")
_lock = threading.Lock()
_lib = None

STATUS = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED", 3: "PKV_ERR_WORKSPACE",
          4: "PKV_ERR_CUDA", 5: "PKV_ERR_DEVICE_RANGE", 6: "PKV_ERR_TIMEOUT"}
F16, BF16, F32 = 0, 1, 2
KV_NATIVE, KV_FP8_E4M3 = 0, 1

# Every symbol include/pkv.h declares.
EXPORTS = ("pkv_kv_cache_append", "pkv_decode_workspace_size", "pkv_decode_split_tokens", "pkv_paged_attn_decode",
           "pkv_paged_attn_decode_step", "pkv_paged_attn_decode_noalloc", "pkv_paged_attn_prefill", "pkv_paged_attn_mixed", "pkv_attn_combine",
           "pkv_rope_append", "pkv_paged_attn_tree", "pkv_tree_workspace_size", "pkv_kv_cache_compact",
           "pkv_get_device_error", "pkv_selftest_wait_timeout", "pkv_status_string", "pkv_version")
DECODE_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024   # PKV_DECODE_NOALLOC_SCRATCH_BYTES in include/pkv.h


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (where, STATUS.get(status, "unknown"), status))


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("inv_freq", ctypes.c_void_p),
                ("mscale", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("block_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("format", ctypes.c_int), ("scales", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libpkv.so (built in-tree by paged_kv_flash_cache_gb300.build). Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libpkv.so is not built (%s); run `python -m paged_kv_flash_cache_gb300.build` or "
                               "__graft_entry__.build()" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.pkv_kv_cache_append.argtypes = [_Cache, P, P, P, P, P, I, I, I, P]
        lib.pkv_kv_cache_append.restype = I
        lib.pkv_decode_workspace_size.argtypes = [I, I, I, I, I, I, I]
        lib.pkv_decode_workspace_size.restype = Z
        lib.pkv_decode_split_tokens.argtypes = [I, I, I, I, I, I, I]
        lib.pkv_decode_split_tokens.restype = I
        lib.pkv_paged_attn_decode.argtypes = [_Cache, P, I, P, P, I, I, F, I, P, Z, P, I, P, P]
        lib.pkv_paged_attn_decode.restype = I
        lib.pkv_paged_attn_decode_step.argtypes = [_Cache, P, I, P, P, I, I, F, I, P, Z, P, I, P, P, P, P]
        lib.pkv_paged_attn_decode_step.restype = I
        lib.pkv_paged_attn_decode_noalloc.argtypes = [_Cache, P, I, P, P, I, I, F, I, P, I, P, P]
        lib.pkv_paged_attn_decode_noalloc.restype = I
        lib.pkv_paged_attn_prefill.argtypes = [_Cache, P, I, P, P, P, I, I, I, I, F, I, P, I, P, P]
        lib.pkv_paged_attn_prefill.restype = I
        lib.pkv_paged_attn_mixed.argtypes = [_Cache, P, I, P, P, P, I, I, I, I, F, I, I, P, Z, P, I, P, P]
        lib.pkv_paged_attn_mixed.restype = I
        L = ctypes.c_longlong
        lib.pkv_rope_append.argtypes = [_Cache, _Rope, P, L, I, P, L, P, L, P, P, P, P, I, I, I, P, L, P]
        lib.pkv_rope_append.restype = I
        lib.pkv_tree_workspace_size.argtypes = [I, I, I, I]
        lib.pkv_tree_workspace_size.restype = Z
        lib.pkv_paged_attn_tree.argtypes = [_Cache, P, I, P, I, P, P, P, I, I, I, I, F, P, Z, P, I, P, P]
        lib.pkv_paged_attn_tree.restype = I
        lib.pkv_kv_cache_compact.argtypes = [_Cache, P, P, P, P, I, I, I, P]
        lib.pkv_kv_cache_compact.restype = I
        lib.pkv_attn_combine.argtypes = [P, P, I, I, I, P, I, P, P]
        lib.pkv_attn_combine.restype = I
        lib.pkv_selftest_wait_timeout.argtypes = [ctypes.c_uint, P]
        lib.pkv_selftest_wait_timeout.restype = I
        lib.pkv_get_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
        lib.pkv_get_device_error.restype = I
        lib.pkv_status_string.argtypes = [I]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_version.argtypes = []
        lib.pkv_version.restype = I
        _lib = lib
        return lib


# ---------------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------------

# A call of a few microseconds on the GPU waits for its marshalling: the helpers take plain ints (ctypes makes the
# pointers), look names up once and enter a device context only when another device is current.

_torch_module = None
_DTYPES = {}
_current_raw_stream = None
_current_device = None


def _torch():
    global _torch_module, _current_raw_stream, _current_device
    if _torch_module is None:
        import torch
        _DTYPES.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        # the current stream's handle without a Stream object around it, where this PyTorch offers it
        _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # (torch.cuda.current_device without its initialisation check, which a CUDA tensor has passed)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _torch_module = torch
    return _torch_module


def _dtype_code(dt) -> int:
    _torch()
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError("unsupported dtype %s" % dt)
    return code


def _dev(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (there is no CPU path)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _i32(t, name):
    if t.dtype != _torch().int32:
        raise TypeError("%s must be int32" % name)
    return _dev(t, name)


def _stream(stream, device=None):
    """The stream's handle; None: the current stream (of device index `device`, or of the current device)."""
    if stream is None:
        torch = _torch()
        if _current_raw_stream is not None:
            return _current_raw_stream(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_device(index, fn, *args):
    """fn(*args) with device `index` current: the library launches on the current device."""
    if _current_device() == index:
        return fn(*args)
    with _torch().cuda.device(index):
        return fn(*args)


def _new(like, shape, dtype, stream):
    """An empty tensor on the device of `like`, from the memory of the stream that the call runs on: work that is still
    pending on another stream never meets it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)  # (new_empty: 3 us more between two launches)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def is_fp8_cache(cache) -> bool:
    torch = _torch()
    dt = cache.dtype
    return dt is torch.uint8 or dt is torch.float8_e4m3fn


def _cache_struct(cache, act_dtype, scales=None) -> _Cache:
    """The C view of `cache`; act_dtype is the type of q / k_new / v_new."""
    torch = _torch_module or _torch()
    shape = cache.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError("cache must be [num_blocks, 2, num_kv_heads, block_size, head_dim]")
    nb, _, hkv, bs, d = shape
    code = _DTYPES.get(cache.dtype)
    if code is not None and scales is None and act_dtype is cache.dtype:
        return _Cache(_dev(cache, "cache"), nb, hkv, bs, d, code, KV_NATIVE, None)
    if is_fp8_cache(cache):
        if scales is None or scales.dtype != torch.float32 or tuple(scales.shape) != (nb, 2, hkv, bs):
            raise ValueError("an FP8 cache needs float32 scales [num_blocks, 2, num_kv_heads, block_size]")
        return _Cache(_dev(cache, "cache"), nb, hkv, bs, d, _dtype_code(act_dtype), KV_FP8_E4M3,
                      _dev(scales, "scales"))
    if scales is not None:
        raise ValueError("scales are only for an FP8 cache")
    if act_dtype != cache.dtype:
        raise TypeError("q / k_new / v_new must have the cache dtype")
    return _Cache(_dev(cache, "cache"), nb, hkv, bs, d, _dtype_code(cache.dtype), KV_NATIVE, None)


def _check(status: int, where: str):
    if status != 0:
        raise PkvError(status, where)


# ---------------------------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------------------------

def kv_cache_append(cache, k_new, v_new, cu_new_lens, ctx_before, block_tables, stream=None, scales=None) -> None:
    """Scatter new tokens' K/V ([T_new, Hkv, D], packed by sequence) into their pages (an FP8
    cache: quantised, with their row scales written to `scales`)."""
    lib = load_library()
    if k_new.dtype != v_new.dtype or k_new.shape != v_new.shape:
        raise TypeError("k_new / v_new must match each other")
    c = _cache_struct(cache, k_new.dtype, scales)
    batch, mb = block_tables.shape
    _check(lib.pkv_kv_cache_append(c, _dev(k_new, "k_new"), _dev(v_new, "v_new"), _i32(cu_new_lens, "cu_new_lens"),
                                   _i32(ctx_before, "ctx_before"), _i32(block_tables, "block_tables"), batch, mb,
                                   int(k_new.shape[0]), _stream(stream)), "pkv_kv_cache_append")


def decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                          num_splits=0) -> int:
    return int(load_library().pkv_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                                        max_blocks_per_seq, num_splits))


def decode_split_tokens(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                        num_splits=0) -> int:
    return int(load_library().pkv_decode_split_tokens(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                                      max_blocks_per_seq, num_splits))


def paged_attn_decode(cache, q, block_tables, context_lens, scale: Optional[float] = None, num_splits: int = 0,
                      workspace=None, out=None, out_dtype=None, lse=None, stream=None, scales=None):
    """One query per sequence ([B, Hq, D]) against its paged context. Returns `out`."""
    torch = _torch()
    lib = load_library()
    c = _cache_struct(cache, q.dtype, scales)
    batch, hq, d = q.shape
    mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((batch, hq, d), dtype=out_dtype or q.dtype, device=q.device)
    need = decode_workspace_size(batch, hq, cache.shape[2], d, cache.shape[3], mb, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    _check(lib.pkv_paged_attn_decode(c, _dev(q, "q"), hq, _i32(block_tables, "block_tables"),
                                     _i32(context_lens, "context_lens"), batch, mb, scale, int(num_splits),
                                     _dev(workspace, "workspace"), ws_bytes, _dev(out, "out"),
                                     _dtype_code(out.dtype), _dev(lse, "lse"), _stream(stream)),
           "pkv_paged_attn_decode")
    return out


def paged_attn_decode_step(cache, q, block_tables, context_lens, k_new, v_new, scale: Optional[float] = None,
                           num_splits: int = 0, workspace=None, out=None, out_dtype=None, lse=None, stream=None,
                           scales=None):
    """One decode step: paged_attn_decode over context_lens[b] cached tokens, and the step's new
    token (k_new / v_new [B, Hkv, D]) written at position context_lens[b]. Returns `out`."""
    torch = _torch()
    lib = load_library()
    if k_new.dtype != q.dtype or v_new.dtype != q.dtype or k_new.shape != v_new.shape:
        raise TypeError("k_new / v_new must match each other and q's dtype")
    c = _cache_struct(cache, q.dtype, scales)
    batch, hq, d = q.shape
    if tuple(k_new.shape) != (batch, cache.shape[2], d):
        raise ValueError("k_new / v_new must be [batch, num_kv_heads, head_dim]")
    mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((batch, hq, d), dtype=out_dtype or q.dtype, device=q.device)
    need = decode_workspace_size(batch, hq, cache.shape[2], d, cache.shape[3], mb, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    _check(lib.pkv_paged_attn_decode_step(c, _dev(q, "q"), hq, _i32(block_tables, "block_tables"),
                                          _i32(context_lens, "context_lens"), batch, mb, scale, int(num_splits),
                                          _dev(workspace, "workspace"), ws_bytes, _dev(out, "out"),
                                          _dtype_code(out.dtype), _dev(lse, "lse"), _dev(k_new, "k_new"),
                                          _dev(v_new, "v_new"), _stream(stream)),
           "pkv_paged_attn_decode_step")
    return out


def paged_attn_decode_noalloc(cache, q, block_tables, context_lens, scale: Optional[float] = None,
                              num_splits: int = 0, out=None, out_dtype=None, lse=None, stream=None, scales=None):
    """paged_attn_decode without a workspace: for callers that cannot allocate device memory.
    The split partials go to a fixed array the library holds on each device (see
    include/pkv.h); sizes needing more than DECODE_NOALLOC_SCRATCH_BYTES raise PkvError
    (PKV_ERR_WORKSPACE). Calls sharing a device must not overlap on the GPU. Returns `out`
    (allocated here with PyTorch only when the caller passes none)."""
    torch = _torch()
    lib = load_library()
    c = _cache_struct(cache, q.dtype, scales)
    batch, hq, d = q.shape
    mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((batch, hq, d), dtype=out_dtype or q.dtype, device=q.device)
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    _check(lib.pkv_paged_attn_decode_noalloc(c, _dev(q, "q"), hq, _i32(block_tables, "block_tables"),
                                             _i32(context_lens, "context_lens"), batch, mb, scale, int(num_splits),
                                             _dev(out, "out"), _dtype_code(out.dtype), _dev(lse, "lse"),
                                             _stream(stream)), "pkv_paged_attn_decode_noalloc")
    return out


def paged_attn_prefill(cache, q, cu_q_lens, context_lens, block_tables, max_q_len: int,
                       scale: Optional[float] = None, causal: bool = True, out=None, out_dtype=None, lse=None,
                       stream=None, scales=None):
    """A chunk of queries per sequence ([sum q_len, Hq, D]) against its paged context
    (the chunk's own K/V already appended). Returns `out`. An FP8 cache (pass `scales`) needs
    head_dim 128; with head_dim 64 it raises PkvError (PKV_ERR_UNSUPPORTED)."""
    torch = _torch()
    lib = load_library()
    c = _cache_struct(cache, q.dtype, scales)
    total_q, hq, d = q.shape
    batch, mb = block_tables.shape
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=out_dtype or q.dtype, device=q.device)
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    _check(lib.pkv_paged_attn_prefill(c, _dev(q, "q"), hq, _i32(cu_q_lens, "cu_q_lens"),
                                      _i32(context_lens, "context_lens"), _i32(block_tables, "block_tables"), batch,
                                      mb, total_q, int(max_q_len), scale, 1 if causal else 0, _dev(out, "out"),
                                      _dtype_code(out.dtype), _dev(lse, "lse"), _stream(stream)),
           "pkv_paged_attn_prefill")
    return out


def paged_attn_mixed(cache, q, cu_q_lens, context_lens, block_tables, max_q_len: int,
                     scale: Optional[float] = None, causal: bool = True, num_splits: int = 0, workspace=None,
                     out=None, out_dtype=None, lse=None, stream=None, scales=None):
    """One call over a batch mixing decode rows (q_len 1) and prefill chunks (q_len > 1):
    q [sum q_len, Hq, D], rows by cu_q_lens. Returns `out`."""
    torch = _torch()
    lib = load_library()
    c = _cache_struct(cache, q.dtype, scales)
    total_q, hq, d = q.shape
    batch, mb = block_tables.shape
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=out_dtype or q.dtype, device=q.device)
    need = decode_workspace_size(batch, hq, cache.shape[2], d, cache.shape[3], mb, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    _check(lib.pkv_paged_attn_mixed(c, _dev(q, "q"), hq, _i32(cu_q_lens, "cu_q_lens"), _i32(context_lens, "context_lens"),
                                    _i32(block_tables, "block_tables"), batch, mb, total_q, int(max_q_len), scale,
                                    1 if causal else 0, int(num_splits), _dev(workspace, "workspace"), ws_bytes,
                                    _dev(out, "out"), _dtype_code(out.dtype), _dev(lse, "lse"), _stream(stream)),
           "pkv_paged_attn_mixed")
    return out


def _at(t, dtype, index, name):
    """Pointer of a contiguous tensor of `dtype` on the cache's device (None: NULL)."""
    if t is None:
        return None
    if t.get_device() != index:
        raise ValueError("%s is on %s, the cache on another device" % (name, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, total, heads, head_dim, dtype, index, name):
    """Pointer and token stride (elements) of [total, heads, head_dim] rows whose tokens may be strided."""
    if t.get_device() != index:
        raise ValueError("%s is on %s, the cache on another device" % (name, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    if t.shape != (total, heads, head_dim):
        raise ValueError("%s must be [%d, %d, %d]" % (name, total, heads, head_dim))
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != head_dim and heads > 1):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    return t.data_ptr(), s0 if total > 1 else heads * head_dim


def rope_append(cache, q, k, v, inv_freq, cu_new_lens, ctx_before, block_tables, positions, interleaved: bool = False,
                mscale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, stream=None,
                scales=None):
    """Norm (with q_weight / k_weight) and rotate the query and key heads of new tokens, write keys and values into
    their pages as kv_cache_append does, and return the rotated queries [T, Hq, D].

    q [T, Hq, D], k and v [T, Hkv, D]: the heads of a token contiguous, tokens at any stride of whole 16 bytes (views
    of one fused projection). inv_freq: float32 [rotary_dim / 2], see `rope.rope_frequencies`; the first
    2 * len(inv_freq) elements of each head are rotated, in pairs (i, i + rotary_dim / 2) or, interleaved,
    (2i, 2i + 1). positions: int32 [T]. q_out: where the queries go (q itself: in place); a new tensor if None."""
    torch = _torch()
    lib = load_library()
    index, dtype, i32 = cache.get_device(), q.dtype, torch.int32
    c = _cache_struct(cache, dtype, scales)
    hkv, d = c.num_kv_heads, c.head_dim
    total, hq = q.shape[0], q.shape[1]
    batch, mb = block_tables.shape
    half = inv_freq.numel()
    if 2 * half > d:
        raise ValueError("inv_freq must be float32 [rotary_dim / 2], rotary_dim <= head_dim")
    if positions.shape != (total,):
        raise ValueError("positions must be [tokens]")
    if cu_new_lens.shape != (batch + 1,) or ctx_before.shape != (batch,):
        raise ValueError("cu_new_lens must be [batch + 1], ctx_before [batch]")
    if (q_weight is not None and q_weight.shape != (d,)) or (k_weight is not None and k_weight.shape != (d,)):
        raise ValueError("q_weight and k_weight must be [head_dim]")
    if scales is not None and scales.get_device() != index:
        raise ValueError("scales on %s, the cache on another device" % scales.device)
    qp, qs = _rows(q, total, hq, d, dtype, index, "q")
    kp, ks = _rows(k, total, hkv, d, dtype, index, "k")
    vp, vs = _rows(v, total, hkv, d, dtype, index, "v")
    if q_out is None:
        q_out = _new(q, (total, hq, d), dtype, stream)
        op, os_ = q_out.data_ptr(), hq * d
    else:
        op, os_ = _rows(q_out, total, hq, d, dtype, index, "q_out")
    rope = _Rope(2 * half, 1 if interleaved else 0, _at(inv_freq, torch.float32, index, "inv_freq"), mscale,
                 _at(q_weight, dtype, index, "q_weight"), _at(k_weight, dtype, index, "k_weight"), eps)
    _check(_on_device(index, lib.pkv_rope_append, c, rope, qp, qs, hq, kp, ks, vp, vs, _at(positions, i32, index, "positions"),
                      _at(cu_new_lens, i32, index, "cu_new_lens"), _at(ctx_before, i32, index, "ctx_before"),
                      _at(block_tables, i32, index, "block_tables"), batch, mb, total, op, os_, _stream(stream, index)),
           "pkv_rope_append")
    return q_out


def tree_workspace_size(num_q_heads, num_kv_heads, head_dim, max_q_len) -> int:
    return int(load_library().pkv_tree_workspace_size(num_q_heads, num_kv_heads, head_dim, max_q_len))


def paged_attn_tree(cache, q, tree_mask, cu_q_lens, context_lens, block_tables, max_q_len: int,
                    scale: Optional[float] = None, workspace=None, out=None, out_dtype=None, lse=None, stream=None,
                    scales=None):
    """Drafted tokens ([sum n_b, Hq, D], their K/V already appended as each sequence's last n_b cached tokens) against
    the paged context and, by tree_mask (int32 [sum n_b, words], bit j % 32 of word j / 32: node i sees node j; see
    `workloads.tree_mask`), one another. Returns `out`."""
    torch = _torch()
    lib = load_library()
    index, dtype, i32 = cache.get_device(), q.dtype, torch.int32
    c = _cache_struct(cache, dtype, scales)
    if scales is not None and scales.get_device() != index:
        raise ValueError("scales on %s, the cache on another device" % scales.device)
    total_q, hq, d = q.shape
    batch, mb = block_tables.shape
    if d != c.head_dim:
        raise ValueError("q must have the cache's head_dim")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != total_q:
        raise ValueError("tree_mask must be [rows of q, words]")
    if cu_q_lens.shape != (batch + 1,) or context_lens.shape != (batch,):
        raise ValueError("cu_q_lens must be [batch + 1], context_lens [batch]")
    if out is None:
        out = _new(q, (total_q, hq, d), out_dtype or dtype, stream)
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if lse is not None and lse.shape != (total_q, hq):
        raise ValueError("lse must be float32 [rows of q, Hq]")
    if workspace is None:
        workspace = _new(q, (lib.pkv_tree_workspace_size(hq, c.num_kv_heads, d, max_q_len),), torch.uint8, stream)
    scale = (1.0 / math.sqrt(d)) if scale is None else float(scale)
    out_code = _dtype_code(out.dtype)
    _check(_on_device(index, lib.pkv_paged_attn_tree, c, _at(q, dtype, index, "q"), hq, _at(tree_mask, i32, index, "tree_mask"),
                      tree_mask.shape[1], _at(cu_q_lens, i32, index, "cu_q_lens"),
                      _at(context_lens, i32, index, "context_lens"), _at(block_tables, i32, index, "block_tables"), batch, mb,
                      total_q, int(max_q_len), scale, _at(workspace, workspace.dtype, index, "workspace"), workspace.nbytes,
                      _at(out, out.dtype, index, "out"), out_code, _at(lse, torch.float32, index, "lse"),
                      _stream(stream, index)), "pkv_paged_attn_tree")
    return out


def kv_cache_compact(cache, keep_pos, cu_keep, dst_start, block_tables, stream=None, scales=None) -> None:
    """Move the cached rows that are kept, in place: row k of sequence b from position keep_pos[cu_keep[b] + k] to
    dst_start[b] + k (every source at or behind its destination). int32: keep_pos [num_keep], cu_keep [batch + 1],
    dst_start [batch]."""
    torch = _torch()
    lib = load_library()
    index, i32 = cache.get_device(), torch.int32
    c = _cache_struct(cache, torch.float16 if scales is not None else cache.dtype, scales)
    batch, mb = block_tables.shape
    if keep_pos.dim() != 1 or cu_keep.shape != (batch + 1,) or dst_start.shape != (batch,):
        raise ValueError("keep_pos must be [num_keep], cu_keep [batch + 1], dst_start [batch]")
    if scales is not None and scales.get_device() != index:
        raise ValueError("scales on %s, the cache on another device" % scales.device)
    _check(_on_device(index, lib.pkv_kv_cache_compact, c, _at(keep_pos, i32, index, "keep_pos"),
                      _at(cu_keep, i32, index, "cu_keep"), _at(dst_start, i32, index, "dst_start"),
                      _at(block_tables, i32, index, "block_tables"), batch, mb, keep_pos.shape[0],
                      _stream(stream, index)), "pkv_kv_cache_compact")


def attn_combine(partial_o, partial_lse, out=None, out_dtype=None, lse=None, stream=None):
    """Merge FP32 split partials [N, S, D] with their lse [N, S]. Returns `out` [N, D]."""
    torch = _torch()
    lib = load_library()
    n, s, d = partial_o.shape
    if out is None:
        out = torch.empty((n, d), dtype=out_dtype or torch.float32, device=partial_o.device)
    _check(lib.pkv_attn_combine(_dev(partial_o, "partial_o"), _dev(partial_lse, "partial_lse"), n, s, d,
                                _dev(out, "out"), _dtype_code(out.dtype), _dev(lse, "lse"), _stream(stream)),
           "pkv_attn_combine")
    return out


def selftest_wait_timeout(timeout_us: int = 20000, stream=None) -> None:
    """Launch one warp that waits on a barrier nothing completes, bounded by timeout_us; the
    device error word then holds PKV_ERR_TIMEOUT (read it with get_device_error)."""
    _check(load_library().pkv_selftest_wait_timeout(int(timeout_us), _stream(stream)), "pkv_selftest_wait_timeout")


def get_device_error(stream=None) -> int:
    """Synchronise the stream, then read and clear the device error word (0 = none)."""
    lib = load_library()
    code = ctypes.c_int(0)
    _check(lib.pkv_get_device_error(_stream(stream), ctypes.byref(code)), "pkv_get_device_error")
    return int(code.value)
