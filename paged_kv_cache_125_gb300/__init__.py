"""GB300-native paged KV-cache attention: the data-parallel hot path of one
attention layer of a nano-vLLM-style serving engine.

Thin Python binding over the C ABI of ``libkvpaged.so`` (declared in
``include/kvpaged.h``).  Every function here only checks and marshals torch
tensors (device pointers, strides, the current CUDA stream) and calls the
library; all the work runs in the library's CUDA kernels.  There is no CPU or
PyTorch fallback: if the library cannot be loaded, every call raises.

    kv_store(k, v, slot_mapping, k_cache, v_cache)
    kv_copy_blocks(kv_cache, block_mapping)
    attn_prefill_varlen(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, ...)
    attn_prefill_varlen_append(q, k, v, slot_mapping, cu_seqlens_q, cu_seqlens_k, ...)
    attn_decode_paged(q, k_cache, v_cache, block_tables, context_lens, max_context_len, ...)
    attn_shared_plan(block_tables, context_lens, ...) + attn_decode_shared(q, ..., plan)
    kv_pages_fork / kv_pages_extend / kv_pages_compact(..., block_tables, context_lens, ref_counts, ...)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
import warnings

__all__ = ["kv_store", "kv_copy_blocks", "attn_prefill_varlen", "attn_prefill_varlen_append",
           "attn_mixed_step",
           "attn_decode_paged", "attn_decode_workspace_size", "attn_decode_paged_noalloc",
           "attn_decode_paged_append",
           "attn_shared_plan", "attn_shared_plan_size", "attn_decode_shared",
           "attn_decode_shared_append", "attn_decode_shared_workspace_size",
           "kv_pages_fork", "kv_pages_extend", "kv_pages_compact", "kv_pages_workspace_size",
           "device_status", "selftest_wait", "library", "library_path", "KvpError"]

_LIB_LOCK = threading.Lock()
_LIB = None

KVP_OK = 0
ERROR_NAMES = {-1: "KVP_ERR_INVALID_ARG", -2: "KVP_ERR_UNSUPPORTED", -3: "KVP_ERR_WORKSPACE",
               -4: "KVP_ERR_CUDA", -5: "KVP_ERR_DEVICE_TIMEOUT", -6: "KVP_ERR_DEVICE_DATA"}

# Every symbol include/kvpaged.h declares, with its ctypes signature.
_P, _I64, _I32, _F32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "kvp_last_error": (ctypes.c_char_p, []),
    "kvp_version": (_I32, []),
    "kvp_device_status": (_I32, []),
    "kvp_selftest_wait": (_I32, [_I32, _P]),
    "kv_store": (_I32, [_P, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P]),
    "kv_copy_blocks": (_I32, [_P, _I64, _I64, _I64, _I64, _P, _I64, _P]),
    "attn_prefill_varlen": (_I32, [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I32, _P, _I32,
                                   _P, _P, _I32, _I32, _I32, _P, _I32, _I32, _I32, _F32, _P, _I64,
                                   _P]),
    "attn_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "attn_decode_paged": (_I32, [_P, _I64, _P, _P, _I64, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32,
                                 _I32, _F32, _P, _SZ, _P, _I64, _P]),
    "attn_decode_paged_noalloc": (_I32, [_P, _I64, _P, _P, _I64, _I32, _P, _I32, _P, _I32, _I32, _I32,
                                         _I32, _I32, _F32, _P, _I64, _P]),
    "attn_decode_paged_append": (_I32, [_P, _I64, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I32, _P, _I32,
                                        _P, _I32, _I32, _I32, _I32, _I32, _F32, _P, _SZ, _P, _I64, _P]),
    "attn_prefill_varlen_append": (_I32, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _I64, _I32, _P, _I32,
                                          _P, _P, _I32, _I32, _I32, _P, _I32, _I32, _I32, _F32, _P, _I64,
                                          _P]),
    "attn_mixed_step": (_I32, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _P, _I64, _I32, _P, _I32, _P, _P,
                               _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _SZ, _P, _I64,
                               _P]),
    "attn_shared_plan_size": (_SZ, [_I32, _I32, _I32]),
    "attn_shared_plan": (_I32, [_P, _I32, _P, _I32, _I64, _I32, _I32, _I32, _I32, _P, _SZ, _P]),
    "attn_decode_shared_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "attn_decode_shared": (_I32, [_P, _I64, _P, _P, _I64, _I32, _P, _I32, _P, _SZ, _I32, _I32, _I32,
                                  _I32, _F32, _P, _SZ, _P, _I64, _P]),
    "attn_decode_shared_append": (_I32, [_P, _I64, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I32, _P, _I32,
                                         _P, _SZ, _I32, _I32, _I32, _I32, _F32, _P, _SZ, _P, _I64, _P]),
    "kv_pages_workspace_size": (_SZ, [_I64, _I32]),
    "kv_pages_fork": (_I32, [_P, _I64, _I64, _I64, _I32, _I64, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P,
                             _P, _P, _SZ, _P]),
    "kv_pages_extend": (_I32, [_P, _I32, _P, _I32, _P, _I64, _I32, _P, _I64, _P, _P, _P, _P, _P, _SZ,
                               _P]),
    "kv_pages_compact": (_I32, [_P, _I64, _I64, _I64, _I32, _I64, _P, _I32, _P, _I32, _P, _P, _P, _P,
                                _P, _SZ, _P]),
}


class KvpError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


def library_path() -> str:
    from . import _build
    return _build.LIB


def library():
    """Loads libkvpaged.so (built by ``__graft_entry__.build()`` or
    ``python -m paged_kv_cache_125_gb300._build``).  Raises if it is missing."""
    global _LIB
    with _LIB_LOCK:
        if _LIB is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"libkvpaged.so is not built ({path}); run "
                                   "`python -m paged_kv_cache_125_gb300._build` first")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype, f.argtypes = res, args
            _LIB = lib
    return _LIB


def _check(rc: int):
    if rc != KVP_OK:
        msg = library().kvp_last_error().decode(errors="replace")
        raise KvpError(rc, msg)


def _stream(t):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, name, dtype, ndim=None, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")


def _rows(t, name, heads, dim):
    """[tokens, heads, dim] with contiguous (heads, dim) -> row stride in elements."""
    if t.shape[1:] != (heads, dim):
        raise ValueError(f"{name} must be [*, {heads}, {dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or t.stride(1) != dim:
        raise ValueError(f"{name}: each token row [heads, head_dim] must be contiguous")
    return t.stride(0)


def _cache_dims(k_cache, v_cache):
    import torch
    _require(k_cache, "k_cache", torch.bfloat16, 4)
    _require(v_cache, "v_cache", torch.bfloat16, 4, k_cache.device)
    if k_cache.shape != v_cache.shape or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("k_cache / v_cache must be contiguous [num_blocks, block_size, kv_heads, head_dim]")
    return k_cache.shape


def device_status() -> int:
    """Reads and clears the device status word (synchronizes)."""
    return int(library().kvp_device_status())


def selftest_wait(arrive: bool, stream=None) -> None:
    """Launches the bounded-wait self-test on the current device: one thread
    waits 2 ms at most on a barrier that it arrives on first (arrive=True) or
    that nothing arrives on (the wait expires and KVP_ERR_DEVICE_TIMEOUT is
    recorded).  Read the outcome with device_status()."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(library().kvp_selftest_wait(1 if arrive else 0, ctypes.c_void_p(s.cuda_stream)))


def kv_store(k, v, slot_mapping, k_cache, v_cache) -> None:
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    _require(k, "k", torch.bfloat16, 3, k_cache.device)
    _require(v, "v", torch.bfloat16, 3, k_cache.device)
    _require(slot_mapping, "slot_mapping", torch.int32, 1, k_cache.device)
    n = slot_mapping.shape[0]
    if k.shape[0] != n or v.shape[0] != n or not slot_mapping.is_contiguous():
        raise ValueError("k, v, slot_mapping must agree on the token count")
    ks, vs = _rows(k, "k", hkv, d), _rows(v, "v", hkv, d)
    _check(library().kv_store(_ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), n, _ptr(k_cache),
                              _ptr(v_cache), nb, bs, hkv, d, _stream(k_cache)))


def kv_copy_blocks(kv_cache, block_mapping) -> None:
    """Copy-on-write block copies in every plane of ``kv_cache``.

    ``kv_cache`` is the engine's cache tensor ``[..., num_blocks, block_size,
    num_kv_heads, head_dim]`` (bf16, contiguous; every leading index, e.g. k/v
    and layer, is one plane).  ``block_mapping`` is ``[n, 2]`` int32 (src, dst)
    on the same device."""
    import torch
    if kv_cache.dtype != torch.bfloat16 or not kv_cache.is_cuda or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous bf16 CUDA tensor")
    if kv_cache.dim() < 4:
        raise ValueError("kv_cache must be [..., num_blocks, block_size, num_kv_heads, head_dim]")
    _require(block_mapping, "block_mapping", torch.int32, 2, kv_cache.device)
    if block_mapping.shape[1] != 2 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous [n, 2] tensor")
    nb = kv_cache.shape[-4]
    block_elems = kv_cache.shape[-3] * kv_cache.shape[-2] * kv_cache.shape[-1]
    planes = kv_cache.numel() // (nb * block_elems)
    _check(library().kv_copy_blocks(_ptr(kv_cache), planes, nb * block_elems, nb, block_elems,
                                    _ptr(block_mapping), block_mapping.shape[0], _stream(kv_cache)))


def attn_decode_workspace_size(num_seqs, num_heads, head_dim, max_context_len, block_size) -> int:
    n = library().attn_decode_workspace_size(num_seqs, num_heads, head_dim, max_context_len, block_size)
    if n == 0 and num_seqs > 0:
        _check(-1)
    return int(n)


def attn_decode_paged(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                      softmax_scale: float | None = None, workspace=None, out=None):
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require(q, "q", torch.bfloat16, 3, dev)
    b, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    if block_tables.shape[0] != b or context_lens.shape[0] != b:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    if not block_tables.is_contiguous() or not context_lens.is_contiguous():
        raise ValueError("block_tables / context_lens must be contiguous")
    if out is None:
        out = torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 3, dev)
    os_ = _rows(out, "out", hq, d)
    need = attn_decode_workspace_size(b, hq, d, max_context_len, bs)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_decode_paged(
        _ptr(q), qs, _ptr(k_cache), _ptr(v_cache), nb, bs, _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), b, int(max_context_len), hq, hkv, d, scale,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), os_,
        _stream(k_cache)))
    return out


def attn_decode_paged_append(q, k, v, slot_mapping, k_cache, v_cache, block_tables, context_lens,
                             max_context_len: int, softmax_scale: float | None = None, workspace=None,
                             out=None):
    """kv_store(k, v, slot_mapping, k_cache, v_cache) followed by
    attn_decode_paged(q, ...), in one launch (see include/kvpaged.h).  Row b
    of k / v is sequence b's new token, stored at slot_mapping[b] (the slot
    of its position context_lens[b] - 1; -1 = padding row)."""
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require(q, "q", torch.bfloat16, 3, dev)
    _require(k, "k", torch.bfloat16, 3, dev)
    _require(v, "v", torch.bfloat16, 3, dev)
    _require(slot_mapping, "slot_mapping", torch.int32, 1, dev)
    b, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    ks, vs = _rows(k, "k", hkv, d), _rows(v, "v", hkv, d)
    if k.shape[0] != b or v.shape[0] != b or slot_mapping.shape[0] != b:
        raise ValueError("k, v and slot_mapping must have one row per sequence")
    if not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous")
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    if block_tables.shape[0] != b or context_lens.shape[0] != b:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    if not block_tables.is_contiguous() or not context_lens.is_contiguous():
        raise ValueError("block_tables / context_lens must be contiguous")
    if out is None:
        out = torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 3, dev)
    os_ = _rows(out, "out", hq, d)
    need = attn_decode_workspace_size(b, hq, d, max_context_len, bs)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_decode_paged_append(
        _ptr(q), qs, _ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), nb,
        bs, _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), b, int(max_context_len),
        hq, hkv, d, scale, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        os_, _stream(k_cache)))
    return out


def attn_decode_paged_noalloc(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                              out, softmax_scale: float | None = None):
    """attn_decode_paged without a workspace: the library's built-in scratch
    is used (see include/kvpaged.h for who needs this and its limits).  The
    caller passes ``out`` ([num_seqs, num_heads, head_dim] bf16): like the
    entry point, this wrapper allocates no device memory."""
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require(q, "q", torch.bfloat16, 3, dev)
    b, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    _require(context_lens, "context_lens", torch.int32, 1, dev)
    if block_tables.shape[0] != b or context_lens.shape[0] != b:
        raise ValueError("block_tables / context_lens must have one row per sequence")
    if not block_tables.is_contiguous() or not context_lens.is_contiguous():
        raise ValueError("block_tables / context_lens must be contiguous")
    _require(out, "out", torch.bfloat16, 3, dev)
    if out.shape[0] != b:
        raise ValueError("out must have one row per sequence")
    os_ = _rows(out, "out", hq, d)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_decode_paged_noalloc(
        _ptr(q), qs, _ptr(k_cache), _ptr(v_cache), nb, bs, _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), b, int(max_context_len), hq, hkv, d, scale,
        _ptr(out), os_, _stream(k_cache)))
    return out


def attn_prefill_varlen(q, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                        k=None, v=None, k_cache=None, v_cache=None, block_tables=None,
                        num_kv_heads: int | None = None, positions=None,
                        softmax_scale: float | None = None, out=None):
    """Keys/values come from k_cache/v_cache through block_tables when block_tables
    is given (prefix-cache hit), else from the packed k, v rows."""
    import torch
    dev = q.device
    _require(q, "q", torch.bfloat16, 3)
    tq, hq, d = q.shape
    qs = _rows(q, "q", hq, d)
    _require(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    _require(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, dev)
    nseq = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != nseq + 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k lengths differ")
    if block_tables is not None:
        nb, bs, hkv, d2 = _cache_dims(k_cache, v_cache)
        if d2 != d:
            raise ValueError("head_dim of q and caches differ")
        _require(block_tables, "block_tables", torch.int32, 2, dev)
        if block_tables.shape[0] != nseq or not block_tables.is_contiguous():
            raise ValueError("block_tables must be contiguous [num_seqs, max_blocks]")
        kp = vp = None
        kvs = tk = 0
        kc, vc, mb = k_cache, v_cache, block_tables.shape[1]
    else:
        _require(k, "k", torch.bfloat16, 3, dev)
        _require(v, "v", torch.bfloat16, 3, dev)
        hkv = k.shape[1] if num_kv_heads is None else num_kv_heads
        kvs = _rows(k, "k", hkv, d)
        if _rows(v, "v", hkv, d) != kvs:
            raise ValueError("k and v must share a row stride")
        kp, vp, kc, vc, nb, bs, mb = k, v, None, None, 0, 16, 0
        tk = k.shape[0]
        if v.shape[0] != tk:
            raise ValueError("k and v must have the same number of rows")
    if out is None:
        out = torch.empty((tq, hq, d), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 3, dev)
    os_ = _rows(out, "out", hq, d)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_prefill_varlen(
        _ptr(q), qs, tq, _ptr(kp), _ptr(vp), kvs, tk, _ptr(kc), _ptr(vc), nb, bs,
        _ptr(block_tables), mb,
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q), int(max_seqlen_k), nseq,
        _ptr(positions), hq, hkv, d, scale, _ptr(out), os_, _stream(q)))
    return out


def attn_prefill_varlen_append(q, k, v, slot_mapping, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                               max_seqlen_k: int, k_cache, v_cache, block_tables=None, positions=None,
                               softmax_scale: float | None = None, out=None):
    """kv_store(k, v, slot_mapping, k_cache, v_cache) followed by
    attn_prefill_varlen, in one launch (see include/kvpaged.h).  Row t of
    k / v is the new key / value of query row t; with block_tables the keys
    are read from the caches (paged), without them from k / v (packed, no
    cached prefix)."""
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require(q, "q", torch.bfloat16, 3, dev)
    _require(k, "k", torch.bfloat16, 3, dev)
    _require(v, "v", torch.bfloat16, 3, dev)
    tq, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    kvs = _rows(k, "k", hkv, d)
    if _rows(v, "v", hkv, d) != kvs:
        raise ValueError("k and v must share a row stride")
    _require(slot_mapping, "slot_mapping", torch.int32, 1, dev)
    if k.shape[0] != tq or v.shape[0] != tq or slot_mapping.shape[0] != tq or \
            not slot_mapping.is_contiguous():
        raise ValueError("k, v and slot_mapping must have one (contiguous) row per query row")
    _require(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    _require(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, dev)
    nseq = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != nseq + 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k lengths differ")
    mb = 0
    if block_tables is not None:
        _require(block_tables, "block_tables", torch.int32, 2, dev)
        if block_tables.shape[0] != nseq or not block_tables.is_contiguous():
            raise ValueError("block_tables must be contiguous [num_seqs, max_blocks]")
        mb = block_tables.shape[1]
    if out is None:
        out = torch.empty((tq, hq, d), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 3, dev)
    os_ = _rows(out, "out", hq, d)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_prefill_varlen_append(
        _ptr(q), qs, tq, _ptr(k), _ptr(v), kvs, _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), nb,
        bs, _ptr(block_tables), mb, _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q),
        int(max_seqlen_k), nseq, _ptr(positions), hq, hkv, d, scale, _ptr(out), os_, _stream(q)))
    return out


def attn_mixed_step(q, k, v, slot_mapping, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, k_cache, v_cache, block_tables, num_decode_seqs: int,
                    decode_sms: int = 0, softmax_scale: float | None = None, workspace=None, out=None):
    """A step of prefill chunks and decode rows (the last num_decode_seqs
    sequences, one query row each): kv_store of every new row, then the
    paged varlen prefill over all sequences, with the decode rows run by the
    decode kernel beside the chunks (see include/kvpaged.h)."""
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, name, torch.bfloat16, 3, dev)
    tq, hq = q.shape[0], q.shape[1]
    qs = _rows(q, "q", hq, d)
    kvs = _rows(k, "k", hkv, d)
    if _rows(v, "v", hkv, d) != kvs:
        raise ValueError("k and v must share a row stride")
    _require(slot_mapping, "slot_mapping", torch.int32, 1, dev)
    if k.shape[0] != tq or v.shape[0] != tq or slot_mapping.shape[0] != tq or \
            not slot_mapping.is_contiguous():
        raise ValueError("k, v and slot_mapping must have one (contiguous) row per query row")
    _require(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    _require(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, dev)
    nseq = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != nseq + 1:
        raise ValueError("cu_seqlens_q / cu_seqlens_k lengths differ")
    _require(block_tables, "block_tables", torch.int32, 2, dev)
    if block_tables.shape[0] != nseq or not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous [num_seqs, max_blocks]")
    if out is None:
        out = torch.empty((tq, hq, d), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 3, dev)
    os_ = _rows(out, "out", hq, d)
    need = attn_decode_workspace_size(max(num_decode_seqs, 1), hq, d, int(max_seqlen_k), bs)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    _check(library().attn_mixed_step(
        _ptr(q), qs, tq, _ptr(k), _ptr(v), kvs, _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), nb, bs,
        _ptr(block_tables), block_tables.shape[1], _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q),
        int(max_seqlen_k), nseq, int(num_decode_seqs), int(decode_sms), hq, hkv, d, scale, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), os_, _stream(q)))
    return out


# The calls below run once per layer or step from Python, next to kernels of a
# few microseconds.  Their arguments are checked and marshalled by an extension
# module (csrc/python/calls.cpp), which makes the call when all is well and
# otherwise returns None: then the checks here name the fault.  Where there is no
# extension module for the installed torch, the code here makes every call itself.

_CALLS = None


class _NoCalls:
    """Stands for the extension module where there is none: takes no call."""

    def __getattr__(self, name):
        return lambda *args: None


def _calls():
    """The extension module, built with the library, or what stands for it."""
    global _CALLS
    library()
    with _LIB_LOCK:
        if _CALLS is None:
            _CALLS = _load_calls() or _NoCalls()
    return _CALLS


def _load_calls():
    import importlib.machinery
    import importlib.util
    from . import _build
    path = _build.calls_path()
    if not os.path.exists(path):
        return None
    loader = importlib.machinery.ExtensionFileLoader("_kvpaged_calls", path)
    spec = importlib.util.spec_from_file_location("_kvpaged_calls", path, loader=loader)
    try:
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"the extension module does not load, its calls go through ctypes: {e}")
        return None
    module.set_check(_check)
    return module


def _call(idx, fn, *args):
    """fn(*args, stream) on device idx, the tensors', and its current stream."""
    import torch
    with torch.cuda.device(idx):
        _check(fn(*args, torch.cuda.current_stream(idx).cuda_stream))


def _sized(name, device, *args) -> int:
    """A size query of the library on a device (None: the current one)."""
    import torch
    fn = getattr(library(), name)
    with torch.cuda.device(device) if device is not None else contextlib.nullcontext():
        n = int(fn(*args))
    if n == 0:
        _check(-1)
    return n


def _int32(t, name, shape, dev):
    """An int32 tensor of that shape (None: any size), contiguous, on dev."""
    import torch
    _require(t, name, torch.int32, len(shape), dev)
    if not t.is_contiguous() or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        raise ValueError(f"{name} must be contiguous [{want}], got {tuple(t.shape)}")


def _scratch(t, name, nbytes, dev):
    """The caller's buffer, or a new one."""
    import torch
    if t is None:
        return torch.empty(nbytes(), dtype=torch.uint8, device=dev)
    _require(t, name, torch.uint8, 1, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _heads_rows(t, name, shape, dev):
    """bf16 rows [rows, heads, head_dim], heads and head_dim contiguous -> row stride."""
    import torch
    _require(t, name, torch.bfloat16, 3, dev)
    if t.shape[0] != shape[0]:
        raise ValueError(f"{name} must have one row per sequence")
    return _rows(t, name, shape[1], shape[2])


def attn_shared_plan_size(num_seqs: int, num_heads: int, num_kv_heads: int, device=None) -> int:
    return _sized("attn_shared_plan_size", device, num_seqs, num_heads, num_kv_heads)


def attn_shared_plan(block_tables, context_lens, block_size: int, num_heads: int, num_kv_heads: int,
                     num_blocks: int, min_shared_len: int = 0, plan=None):
    """Finds the leading pages that neighbouring sequences of a decode batch
    share (see include/kvpaged.h) and returns the plan, a uint8 device tensor
    that attn_decode_shared / attn_decode_shared_append of every layer of this
    step take.  ``plan``: a buffer to fill (attn_shared_plan_size bytes)."""
    done = (_CALLS or _calls()).attn_shared_plan(block_tables, context_lens, block_size, num_heads,
                                                 num_kv_heads, num_blocks, min_shared_len, plan)
    if done is not None:
        return done
    import torch
    _require(block_tables, "block_tables", torch.int32, 2)
    dev = block_tables.device
    b, width = block_tables.shape
    _int32(block_tables, "block_tables", (b, width), dev)
    _int32(context_lens, "context_lens", (b,), dev)
    plan = _scratch(plan, "plan", lambda: attn_shared_plan_size(b, num_heads, num_kv_heads, dev), dev)
    _call(dev.index, library().attn_shared_plan, block_tables.data_ptr(), width, context_lens.data_ptr(), b,
          num_blocks, block_size, num_heads, num_kv_heads, min_shared_len, plan.data_ptr(), plan.numel())
    return plan


def attn_decode_shared_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                      device=None) -> int:
    return _sized("attn_decode_shared_workspace_size", device, num_seqs, num_heads, num_kv_heads, head_dim)


def attn_decode_shared(q, k_cache, v_cache, block_tables, plan, softmax_scale: float | None = None,
                       workspace=None, out=None):
    """attn_decode_paged over a batch planned by attn_shared_plan (which has
    the context lengths): the pages that a group of neighbouring sequences
    share are read once for the group."""
    done = (_CALLS or _calls()).attn_decode_shared(q, None, None, None, k_cache, v_cache, block_tables, plan,
                                                   softmax_scale, workspace, out)
    if done is not None:
        return done
    return _decode_shared(q, None, None, None, k_cache, v_cache, block_tables, plan, softmax_scale, workspace,
                          out)


def attn_decode_shared_append(q, k, v, slot_mapping, k_cache, v_cache, block_tables, plan,
                              softmax_scale: float | None = None, workspace=None, out=None):
    """kv_store(k, v, slot_mapping, k_cache, v_cache) followed by
    attn_decode_shared, in one call (see include/kvpaged.h).  Row b of k / v
    is sequence b's new token, stored at slot_mapping[b]."""
    if k is None:
        raise TypeError("k must be a torch.Tensor")
    done = (_CALLS or _calls()).attn_decode_shared(q, k, v, slot_mapping, k_cache, v_cache, block_tables, plan,
                                                   softmax_scale, workspace, out)
    if done is not None:
        return done
    return _decode_shared(q, k, v, slot_mapping, k_cache, v_cache, block_tables, plan, softmax_scale, workspace,
                          out)


def _decode_shared(q, k, v, slot_mapping, k_cache, v_cache, block_tables, plan, softmax_scale, workspace, out):
    import torch
    nb, bs, hkv, d = _cache_dims(k_cache, v_cache)
    dev = k_cache.device
    _require(q, "q", torch.bfloat16, 3, dev)
    b, hq, _ = q.shape
    if q.shape[2] != d:
        raise ValueError("head_dim of q and caches differ")
    qs = _heads_rows(q, "q", q.shape, dev)
    _int32(block_tables, "block_tables", (b, None), dev)
    if out is None:
        out = torch.empty((b, hq, d), dtype=torch.bfloat16, device=dev)
    os_ = _heads_rows(out, "out", q.shape, dev)
    if plan is None:
        raise TypeError("plan must be a torch.Tensor")
    plan = _scratch(plan, "plan", None, dev)
    workspace = _scratch(workspace, "workspace",
                         lambda: attn_decode_shared_workspace_size(b, hq, hkv, d, dev), dev)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    rest = (k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, block_tables.data_ptr(), block_tables.shape[1],
            plan.data_ptr(), plan.numel(), b, hq, hkv, d, scale, workspace.data_ptr(), workspace.numel(),
            out.data_ptr(), os_)
    if k is None:
        _call(dev.index, library().attn_decode_shared, q.data_ptr(), qs, *rest)
        return out
    new = (b, hkv, d)
    ks, vs = _heads_rows(k, "k", new, dev), _heads_rows(v, "v", new, dev)
    _int32(slot_mapping, "slot_mapping", (b,), dev)
    _call(dev.index, library().attn_decode_shared_append, q.data_ptr(), qs, k.data_ptr(), v.data_ptr(), ks, vs,
          slot_mapping.data_ptr(), *rest)
    return out


def kv_pages_workspace_size(num_blocks: int, num_rows: int) -> int:
    return _sized("kv_pages_workspace_size", None, num_blocks, num_rows)


def _pool_dims(kv_cache):
    """[..., num_blocks, block_size, num_kv_heads, head_dim] -> device,
    planes, plane stride, num_blocks, block_size, row elements."""
    import torch
    if not isinstance(kv_cache, torch.Tensor):
        raise TypeError("kv_cache must be a torch.Tensor")
    if kv_cache.dtype is not torch.bfloat16 or not kv_cache.is_cuda or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous bf16 CUDA tensor")
    if kv_cache.dim() < 4:
        raise ValueError("kv_cache must be [..., num_blocks, block_size, num_kv_heads, head_dim]")
    nb, bs, hkv, d = kv_cache.shape[-4:]
    plane = nb * bs * hkv * d
    return kv_cache.device, kv_cache.numel() // max(plane, 1), plane, nb, bs, hkv * d


def _outputs(out, names, shapes, dev):
    """The caller's output tensors, checked, or new ones."""
    import torch
    if out is None:
        return tuple(torch.empty(s, dtype=torch.int32, device=dev) for s in shapes)
    if len(out) != len(shapes):
        raise ValueError(f"out must be {len(shapes)} tensors")
    for t, name, shape in zip(out, names, shapes):
        _int32(t, name, shape, dev)
    return tuple(out)


def kv_pages_fork(kv_cache, block_tables, context_lens, ref_counts, parents, workspace=None, out=None):
    """New rows from old ones: fork, reorder, free (see include/kvpaged.h).
    Row r of the result continues row parents[r] (-1: an empty row); an
    unfilled last page that several rows would write to is copied in every
    plane of ``kv_cache``.  Returns (block_tables, context_lens, ref_counts):
    new tensors, or ``out``, three tensors that do not overlap the inputs."""
    done = (_CALLS or _calls()).kv_pages_fork(kv_cache, block_tables, context_lens, ref_counts, parents,
                                              workspace, out)
    if done is not None:
        return done
    dev, planes, stride, nb, bs, row = _pool_dims(kv_cache)
    _int32(block_tables, "block_tables", (None, None), dev)
    n, mb = block_tables.shape
    _int32(context_lens, "context_lens", (n,), dev)
    _int32(ref_counts, "ref_counts", (nb,), dev)
    _int32(parents, "parents", (None,), dev)
    m = parents.shape[0]
    out = _outputs(out, ("out tables", "out context_lens", "out ref_counts"), ((m, mb), (m,), (nb,)), dev)
    ws = _scratch(workspace, "workspace", lambda: kv_pages_workspace_size(nb, max(n, m)), dev)
    _call(dev.index, library().kv_pages_fork, kv_cache.data_ptr(), planes, stride, nb, bs, row,
          block_tables.data_ptr(), mb, context_lens.data_ptr(), n, ref_counts.data_ptr(),
          parents.data_ptr(), m, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(),
          ws.data_ptr(), ws.numel())
    return out


def kv_pages_extend(block_tables, context_lens, ref_counts, new_tokens, block_size: int, num_slots: int,
                    workspace=None, out=None):
    """Room for new_tokens[r] more tokens in each row (see
    include/kvpaged.h).  Returns (block_tables, context_lens, ref_counts,
    slot_mapping), slot_mapping [num_slots] holding the new tokens' slots row
    after row, then -1.  ``out``: those four tensors; the first three may be
    the inputs themselves."""
    done = (_CALLS or _calls()).kv_pages_extend(block_tables, context_lens, ref_counts, new_tokens, block_size,
                                                num_slots, workspace, out)
    if done is not None:
        return done
    import torch
    _require(block_tables, "block_tables", torch.int32, 2)
    dev = block_tables.device
    n, mb = block_tables.shape
    _int32(block_tables, "block_tables", (n, mb), dev)
    _int32(context_lens, "context_lens", (n,), dev)
    _int32(ref_counts, "ref_counts", (None,), dev)
    _int32(new_tokens, "new_tokens", (n,), dev)
    nb = ref_counts.shape[0]
    out = _outputs(out, ("out tables", "out context_lens", "out ref_counts", "slot_mapping"),
                   ((n, mb), (n,), (nb,), (num_slots,)), dev)
    ws = _scratch(workspace, "workspace", lambda: kv_pages_workspace_size(nb, n), dev)
    _call(dev.index, library().kv_pages_extend, block_tables.data_ptr(), mb, context_lens.data_ptr(), n,
          ref_counts.data_ptr(), nb, block_size, new_tokens.data_ptr(), num_slots, out[0].data_ptr(),
          out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), ws.data_ptr(), ws.numel())
    return out


def kv_pages_compact(kv_cache, block_tables, context_lens, ref_counts, workspace=None, out=None):
    """Moves the pages in use to the front of the pool, in every plane of
    ``kv_cache`` (see include/kvpaged.h).  Returns (block_tables, ref_counts,
    places), places[p] being the new id of page p (-1 if it was free): new
    tensors, or ``out``, three tensors that do not overlap the inputs."""
    done = (_CALLS or _calls()).kv_pages_compact(kv_cache, block_tables, context_lens, ref_counts, workspace, out)
    if done is not None:
        return done
    dev, planes, stride, nb, bs, row = _pool_dims(kv_cache)
    _int32(block_tables, "block_tables", (None, None), dev)
    n, mb = block_tables.shape
    _int32(context_lens, "context_lens", (n,), dev)
    _int32(ref_counts, "ref_counts", (nb,), dev)
    out = _outputs(out, ("out tables", "out ref_counts", "places"), ((n, mb), (nb,), (nb,)), dev)
    ws = _scratch(workspace, "workspace", lambda: kv_pages_workspace_size(nb, n), dev)
    _call(dev.index, library().kv_pages_compact, kv_cache.data_ptr(), planes, stride, nb, bs, row,
          block_tables.data_ptr(), mb, context_lens.data_ptr(), n, ref_counts.data_ptr(),
          out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(), ws.numel())
    return out
