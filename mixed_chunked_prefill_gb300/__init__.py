"""Mixed chunked-prefill + decode paged attention for GB300 (sm_103a).

Python binding of the C ABI in ``include/mcp.h``.  The functions here only
check and marshal arguments (torch tensors -> device pointers, the current
CUDA stream); every step of the computation runs in the library's CUDA
kernels.  If the library is not built, every call raises: there is no CPU or
PyTorch fallback.
"""

from __future__ import annotations

import ctypes

import numpy as np

from . import _capi
from ._capi import (  # noqa: F401
    DEVERR_ITEM_KIND,
    DEVERR_NO_PAGES,
    DEVERR_PAGE_RANGE,
    DEVERR_PROBS,
    DEVERR_REQUEST,
    DEVERR_ROW_RANGE,
    DEVERR_SEGMENT,
    DEVERR_SLOT_DUP,
    DEVERR_SLOT_RANGE,
    DEVERR_TIMEOUT,
    DEVERR_TOKEN_RANGE,
    DEVERR_TREE,
    AttnDesc,
    MCPError,
    Plan,
    PlanOptions,
    RequestPool,
)

__all__ = [
    "AttnDesc", "Plan", "PlanOptions", "MCPError", "load", "abi_version", "paged_kv_append",
    "build_slot_mapping", "mixed_attn_plan", "mixed_attn_fwd", "check_device_errors",
    "workspace_error_word", "merge_states", "make_desc", "mixed_attn_fwd_noalloc",
    "mixed_attn_plan_rows", "build_logits_indices", "gather_rows", "kv_copy_pages",
    "mixed_attn_varlen", "RequestPool", "make_request_pool", "build_step_tables", "commit_step",
    "mixed_conv", "mixed_scan", "update_token_counts", "process_logits", "build_tree_masks",
    "mixed_attn_fwd_tree", "verify_drafts", "kv_keep_path",
]


def load():
    return _capi.load()


def abi_version() -> int:
    return int(load().mcp_abi_version())


def _stream(stream):
    import torch

    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dev(t, dtype, name):
    import torch

    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host_i32(a, name):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, a.ctypes.data_as(ctypes.c_void_p)


def make_desc(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim, page_size,
              max_pages_per_seq, num_pages, sm_scale) -> AttnDesc:
    return AttnDesc(int(num_seqs), int(total_q), int(num_q_heads), int(num_kv_heads),
                    int(head_dim), int(page_size), int(max_pages_per_seq), int(num_pages),
                    float(sm_scale))


def paged_kv_append(k_new, v_new, slot_mapping, k_cache, v_cache, error_word=None, stream=None):
    """Scatter k_new/v_new [T, H_kv, D] (bf16) into the paged caches
    [num_pages, P, H_kv, D] at slot_mapping [T] (int64; < 0 skips).
    ``error_word``: None, an int32 CUDA tensor, or a device address."""
    import torch

    lib = load()
    T = int(k_new.shape[0]) if k_new.dim() > 0 else 0
    num_pages, P, Hkv, D = (int(x) for x in k_cache.shape)
    if tuple(k_new.shape) != (T, Hkv, D) or tuple(v_new.shape) != (T, Hkv, D):
        raise ValueError("k_new / v_new must be [T, H_kv, D] matching the cache")
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache shapes differ")
    if tuple(slot_mapping.shape) != (T,):
        raise ValueError("slot_mapping must be [T]")
    if error_word is None or isinstance(error_word, torch.Tensor):
        ew = _dev(error_word, torch.int32, "error_word")
    else:  # a device address, e.g. workspace_error_word(plan, workspace)
        ew = ctypes.c_void_p(int(error_word))
    st = lib.mcp_paged_kv_append(
        _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"),
        _dev(slot_mapping, torch.int64, "slot_mapping"), T, Hkv, D, P, num_pages,
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        ew, _stream(stream))
    _capi.check(st, "paged_kv_append")


def build_slot_mapping(block_tables, cu_seqlens_q, seqlens_k, page_size, num_pages) -> np.ndarray:
    """Host-side slot mapping of the step's new tokens (int64 numpy array)."""
    lib = load()
    bt = np.ascontiguousarray(np.asarray(block_tables, dtype=np.int32))
    S = bt.shape[0]
    cu, cu_p = _host_i32(cu_seqlens_q, "cu_seqlens_q")
    sk, sk_p = _host_i32(seqlens_k, "seqlens_k")
    out = np.empty(int(cu[-1]), dtype=np.int64)
    st = lib.mcp_build_slot_mapping(bt.ctypes.data_as(ctypes.c_void_p), S,
                                    bt.shape[1] if bt.ndim == 2 else 0, int(page_size),
                                    int(num_pages), cu_p, sk_p,
                                    out.ctypes.data_as(ctypes.c_void_p))
    _capi.check(st, "build_slot_mapping")
    return out


def mixed_attn_plan(desc: AttnDesc, cu_seqlens_q, seqlens_k, options: PlanOptions | None = None,
                    workspace=None, stream=None) -> Plan:
    """Plan a step from HOST metadata; with ``workspace`` (uint8 CUDA tensor)
    also copy the work lists into it."""
    import torch

    lib = load()
    cu, cu_p = _host_i32(cu_seqlens_q, "cu_seqlens_q")
    sk, sk_p = _host_i32(seqlens_k, "seqlens_k")
    plan = Plan()
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = int(workspace.numel()) if workspace is not None else 0
    st = lib.mcp_mixed_attn_plan(ctypes.byref(desc), cu_p, sk_p,
                                 ctypes.byref(options) if options is not None else None,
                                 ctypes.byref(plan), ws, nbytes,
                                 _stream(stream) if workspace is not None else None)
    _capi.check(st, "mixed_attn_plan")
    return plan


def mixed_attn_plan_rows(desc: AttnDesc, cu_seqlens_q, seqlens_k, rows,
                         options: PlanOptions | None = None, workspace=None,
                         stream=None) -> Plan:
    """Plan attention for the listed query rows only (HOST token indices,
    strictly increasing); with ``workspace`` also copy the work lists into it."""
    import torch

    lib = load()
    cu, cu_p = _host_i32(cu_seqlens_q, "cu_seqlens_q")
    sk, sk_p = _host_i32(seqlens_k, "seqlens_k")
    rw, rw_p = _host_i32(rows, "rows")
    plan = Plan()
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = int(workspace.numel()) if workspace is not None else 0
    st = lib.mcp_mixed_attn_plan_rows(ctypes.byref(desc), cu_p, sk_p, rw_p, int(rw.size),
                                      ctypes.byref(options) if options is not None else None,
                                      ctypes.byref(plan), ws, nbytes,
                                      _stream(stream) if workspace is not None else None)
    _capi.check(st, "mixed_attn_plan_rows")
    return plan


def build_logits_indices(cu_seqlens_q, sample_mask=None) -> np.ndarray:
    """The last token of every segment with a token this step (optionally only
    segments with a non-zero ``sample_mask``): int32 numpy array."""
    lib = load()
    cu, cu_p = _host_i32(cu_seqlens_q, "cu_seqlens_q")
    S = int(cu.size) - 1
    out = np.empty(max(S, 1), dtype=np.int32)
    count = ctypes.c_int32()
    mask_p = None
    if sample_mask is not None:
        m = np.ascontiguousarray(np.asarray(sample_mask, dtype=np.uint8))
        if m.size != S:
            raise ValueError("sample_mask must have one entry per segment")
        mask_p = m.ctypes.data_as(ctypes.c_void_p)
    st = lib.mcp_build_logits_indices(S, cu_p, mask_p, out.ctypes.data_as(ctypes.c_void_p),
                                      ctypes.byref(count))
    _capi.check(st, "build_logits_indices")
    return out[:count.value].copy()


def kv_copy_pages(k_src, v_src, k_dst, v_dst, src_pages, dst_pages, error_word=None,
                  stream=None) -> None:
    """Copy whole KV pages between two pools ([pages, P, H_kv, D] bf16 tensors,
    device or page-locked host): dst[dst_pages[i]] = src[src_pages[i]].
    ``src_pages`` / ``dst_pages``: int32 tensors on the device (or pinned)."""
    import torch

    lib = load()
    n = int(src_pages.numel())
    if int(dst_pages.numel()) != n:
        raise ValueError("src_pages and dst_pages differ in length")
    for t, name in ((k_src, "k_src"), (v_src, "v_src"), (k_dst, "k_dst"), (v_dst, "v_dst")):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 page pool")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be device or page-locked host memory")
    if tuple(k_src.shape[1:]) != tuple(k_dst.shape[1:]) or k_src.shape != v_src.shape \
            or k_dst.shape != v_dst.shape:
        raise ValueError("pools must have the same page shape")
    for t, name in ((src_pages, "src_pages"), (dst_pages, "dst_pages")):
        if t.dtype != torch.int32 or not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be an int32 device (or pinned) tensor")
    page_bytes = int(k_src[0].numel()) * 2
    if error_word is None or isinstance(error_word, torch.Tensor):
        ew = _dev(error_word, torch.int32, "error_word")
    else:
        ew = ctypes.c_void_p(int(error_word))
    st = lib.mcp_kv_copy_pages(ctypes.c_void_p(k_src.data_ptr()), ctypes.c_void_p(v_src.data_ptr()),
                               int(k_src.shape[0]), ctypes.c_void_p(k_dst.data_ptr()),
                               ctypes.c_void_p(v_dst.data_ptr()), int(k_dst.shape[0]), page_bytes,
                               ctypes.c_void_p(src_pages.data_ptr()),
                               ctypes.c_void_p(dst_pages.data_ptr()), n, ew, _stream(stream))
    _capi.check(st, "kv_copy_pages")


def gather_rows(src, rows, dst, error_word=None, stream=None) -> None:
    """dst[i] = src[rows[i]] along the first dimension (device tensors; rows int32)."""
    import torch

    lib = load()
    n = int(rows.numel())
    if dst.shape[0] != n or tuple(dst.shape[1:]) != tuple(src.shape[1:]) or dst.dtype != src.dtype:
        raise ValueError("dst must be [len(rows), *src.shape[1:]] of src's dtype")
    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src / dst must be contiguous CUDA tensors")
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] else dst[0].numel() * dst.element_size()
    if error_word is None or isinstance(error_word, torch.Tensor):
        ew = _dev(error_word, torch.int32, "error_word")
    else:
        ew = ctypes.c_void_p(int(error_word))
    st = lib.mcp_gather_rows(ctypes.c_void_p(src.data_ptr()), int(src.shape[0]), int(row_bytes),
                             _dev(rows, torch.int32, "rows"), n, ctypes.c_void_p(dst.data_ptr()),
                             ew, _stream(stream))
    _capi.check(st, "gather_rows")


def mixed_attn_fwd(plan: Plan, q, k_cache, v_cache, block_tables, cu_seqlens_q, seqlens_k, out,
                   lse=None, workspace=None, stream=None) -> None:
    """Fused mixed attention forward on device tensors (see include/mcp.h)."""
    import torch

    lib = load()
    st = lib.mcp_mixed_attn_fwd(
        ctypes.byref(plan), _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q"), _dev(seqlens_k, torch.int32, "seqlens_k"),
        _dev(out, torch.bfloat16, "out"), _dev(lse, torch.float32, "lse"),
        _dev(workspace, torch.uint8, "workspace"),
        int(workspace.numel()) if workspace is not None else 0, _stream(stream))
    _capi.check(st, "mixed_attn_fwd")


def mixed_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, sm_scale, out=None, lse=None,
                      options: PlanOptions | None = None, stream=None):
    """Right-aligned causal attention over packed non-paged K/V ([W] "Flash
    Attention 的 varlen 接口"): q [T, H_q, D], k / v [total_k, H_kv, D] bf16
    CUDA tensors; cu_seqlens_q / cu_seqlens_k host int arrays.  Plans, runs
    and checks the device error word; returns ``out`` (and fills ``lse``)."""
    import torch

    lib = load()
    cu_q = np.ascontiguousarray(np.asarray(cu_seqlens_q, dtype=np.int32))
    cu_k = np.ascontiguousarray(np.asarray(cu_seqlens_k, dtype=np.int32))
    S = int(cu_q.size) - 1
    if cu_k.size != S + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k differ in length")
    sk = np.diff(cu_k).astype(np.int32)
    T, Hq, D = (int(x) for x in q.shape)
    total_k, Hkv = int(k.shape[0]), int(k.shape[1])
    if int(cu_k[-1]) != total_k or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k / v must be [cu_seqlens_k[-1], H_kv, D]")
    mp = max(1, int((sk.max() + 15) // 16)) if S else 1
    desc = make_desc(S, T, Hq, Hkv, D, 16, mp, 1, sm_scale)
    sizing = mixed_attn_plan(desc, cu_q, sk, options)
    ws = torch.empty(max(256, int(sizing.workspace_bytes)), dtype=torch.uint8, device=q.device)
    plan = mixed_attn_plan(desc, cu_q, sk, options, ws, stream)
    if out is None:
        out = torch.empty_like(q)
    cu_q_d = torch.from_numpy(cu_q).to(q.device)
    cu_k_d = torch.from_numpy(cu_k).to(q.device)
    st = lib.mcp_mixed_attn_fwd_varlen(
        ctypes.byref(plan), _dev(q, torch.bfloat16, "q"), _dev(k, torch.bfloat16, "k"),
        _dev(v, torch.bfloat16, "v"), _dev(cu_q_d, torch.int32, "cu_seqlens_q"),
        _dev(cu_k_d, torch.int32, "cu_seqlens_k"), total_k, _dev(out, torch.bfloat16, "out"),
        _dev(lse, torch.float32, "lse"), _dev(ws, torch.uint8, "workspace"), int(ws.numel()),
        _stream(stream))
    _capi.check(st, "mixed_attn_fwd_varlen")
    check_device_errors(workspace_error_word(plan, ws), stream)
    return out


def workspace_error_word(plan: Plan, workspace) -> int:
    lib = load()
    return int(lib.mcp_workspace_error_word(ctypes.byref(plan), ctypes.c_void_p(workspace.data_ptr())))


def check_device_errors(error_word_ptr: int, stream=None) -> None:
    """Synchronise, read and clear a device error word; raise on a set bit."""
    lib = load()
    st = lib.mcp_check_device_errors(ctypes.c_void_p(int(error_word_ptr)), _stream(stream))
    _capi.check(st, "check_device_errors")


def merge_states(o_parts, lse_parts, out, lse_out=None, stream=None) -> None:
    """Merge split attention states: o_parts [n, R, H, D] fp32, lse_parts [n, R, H]."""
    import torch

    lib = load()
    n, R, H, D = (int(x) for x in o_parts.shape)
    if tuple(lse_parts.shape) != (n, R, H) or tuple(out.shape) != (R, H, D):
        raise ValueError("shape mismatch")
    st = lib.mcp_merge_states(_dev(o_parts, torch.float32, "o_parts"),
                              _dev(lse_parts, torch.float32, "lse_parts"), n, R, H, D,
                              _dev(out, torch.bfloat16, "out"),
                              _dev(lse_out, torch.float32, "lse_out"), _stream(stream))
    _capi.check(st, "merge_states")


def mixed_attn_fwd_noalloc(desc: AttnDesc, h_cu_seqlens_q, h_seqlens_k, q, k_cache, v_cache,
                           block_tables, cu_seqlens_q, seqlens_k, out, lse=None,
                           options: PlanOptions | None = None, stream=None) -> int:
    """Mixed attention forward without a workspace (for callers that cannot
    allocate device memory): plans from the HOST metadata and keeps its scratch
    in the library's fixed 16 MiB device array.  Returns the device address of
    this call's error word (for check_device_errors).  Calls that overlap on
    the GPU race; make the first call on a device before any stream capture."""
    import torch

    lib = load()
    cu, cu_p = _host_i32(h_cu_seqlens_q, "h_cu_seqlens_q")
    sk, sk_p = _host_i32(h_seqlens_k, "h_seqlens_k")
    ew = ctypes.c_void_p()
    st = lib.mcp_mixed_attn_fwd_noalloc(
        ctypes.byref(desc), cu_p, sk_p, ctypes.byref(options) if options is not None else None,
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q"), _dev(seqlens_k, torch.int32, "seqlens_k"),
        _dev(out, torch.bfloat16, "out"), _dev(lse, torch.float32, "lse"), ctypes.byref(ew),
        _stream(stream))
    _capi.check(st, "mixed_attn_fwd_noalloc")
    return int(ew.value or 0)


# ---------------------------------------------------------------------------
# the operators around a step's attention
# ---------------------------------------------------------------------------

# A step makes these calls for every layer or token, so the checks are written
# for the good case: one comparison per property, the message worked out apart.

def _gpu(t, name) -> int:
    """Index of the device that tensor ``t`` is on."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _refuse(t, dtype, name, dev, shape):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, name, dev, shape=None):
    """Device address of a contiguous tensor on device ``dev`` (None: no address)."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, name, dev, shape)


def _row_arg(t, dtype, name, dev, shape):
    """(address, stride between tokens) of [tokens, ...] rows that may be part of wider rows:
    everything behind the first dimension is dense."""
    try:
        good = t.dtype is dtype and t.get_device() == dev and t.shape == shape
    except AttributeError:
        good = False
    if not good:
        _refuse(t, dtype, name, dev, shape)
    strides = t.stride()
    row = 1
    for k in range(len(shape) - 1, 0, -1):
        if shape[k] != 1 and strides[k] != row:
            raise ValueError(f"{name}: a token's row must be dense, got strides {strides}")
        row *= shape[k]
    return t.data_ptr(), strides[0] if shape[0] > 1 else -(-row // 8) * 8


def _sizes(*sizes):
    """The C structures hold 32-bit sizes; a larger one would be cut off, not refused."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"a size of {max(sizes)} is past 32 bits")


def _error(error_word, dev):
    """Address of an error word: None, an int32 CUDA tensor, or a device address."""
    if error_word is None:
        return None
    import torch

    if isinstance(error_word, torch.Tensor):
        return _arg(error_word, torch.int32, "error_word", dev)
    return int(error_word)


def _launch(where, dev, stream, fn, *args):
    """Call ``fn(*args, stream)`` with ``dev`` as the current device."""
    if _current_device is None:
        _bind()
    if dev != _current_device():
        import torch

        with torch.cuda.device(dev):
            return _launch(where, dev, stream, fn, *args)
    if stream is None:
        raw = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    st = fn(*args, raw)
    if st:
        _capi.check(st, where)


def _launch_free(where, dev, fn, *args):
    """Call ``fn(*args)``, which takes no stream, with ``dev`` as the current device."""
    if _current_device is None:
        _bind()
    if dev != _current_device():
        import torch

        with torch.cuda.device(dev):
            return _launch_free(where, dev, fn, *args)
    st = fn(*args)
    if st:
        _capi.check(st, where)


_current_device = _raw_stream = None


def _bind():
    """What a call asks torch for: the current device, and the current stream of a device
    (without a Stream object, where torch allows it)."""
    global _current_device, _raw_stream
    import torch

    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _empty(shape, dtype, device, stream, result=False):
    """A new tensor for a call on ``stream`` (None: the current one): its memory belongs to
    that stream, so that nothing else that is queued can still write it.  ``result``: the
    caller keeps it and may use it on the current stream."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    there = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.stream(there):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result and there.cuda_stream != here.cuda_stream:
        t.record_stream(here)
    return t


def make_request_pool(request_pages, request_lens, free_pages, free_count,
                      page_size) -> RequestPool:
    """The device-side pages of all requests (see ``mcp_request_pool`` in include/mcp.h) over
    int32 CUDA tensors: request_pages [R, max_pages_per_seq], request_lens [R], free_pages
    [num_pages], free_count [1].  The tensors stay the caller's state; the pool keeps them."""
    import torch

    dev = _gpu(request_pages, "request_pages")
    if request_pages.dim() != 2:
        raise ValueError("request_pages must be [max_requests, max_pages_per_seq]")
    R, width = request_pages.shape
    _sizes(R, width, int(page_size), free_pages.numel())
    i32 = torch.int32
    pool = RequestPool(
        R, width, int(page_size), int(free_pages.numel()),
        _arg(request_pages, i32, "request_pages", dev),
        _arg(request_lens, i32, "request_lens", dev, (R,)),
        _arg(free_pages, i32, "free_pages", dev),
        _arg(free_count, i32, "free_count", dev, (1,)))
    pool.tensors = (request_pages, request_lens, free_pages, free_count)
    pool.device = dev
    return pool


def _pool_device(pool, request_ids) -> int:
    dev = _gpu(request_ids, "request_ids")
    if getattr(pool, "device", dev) != dev:
        raise ValueError(f"request_ids must be on cuda:{pool.device}, where the pool is")
    return dev


def build_step_tables(pool: RequestPool, request_ids, q_lens, cu_seqlens_q, seqlens_k,
                      block_tables, slot_mapping, positions=None, logits_indices=None,
                      error_word=None, stream=None) -> None:
    """Tables, slots and pages of a step from the lengths in ``pool`` (see include/mcp.h):
    request_ids, q_lens [S] in; cu_seqlens_q [S + 1], seqlens_k [S], block_tables
    [S, max_pages_per_seq], slot_mapping [max_tokens] (int64), positions [max_tokens] and
    logits_indices [S] out, all int32 CUDA tensors otherwise."""
    import torch

    dev, i32 = _pool_device(pool, request_ids), torch.int32
    S, cap = int(request_ids.shape[0]), int(slot_mapping.shape[0])
    _sizes(S, cap)
    one = (S,)
    _launch("build_step_tables", dev, stream, load().mcp_build_step_tables, ctypes.byref(pool),
            _arg(request_ids, i32, "request_ids", dev, one), _arg(q_lens, i32, "q_lens", dev, one),
            S, cap, _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, one),
            _arg(block_tables, i32, "block_tables", dev, (S, pool.max_pages_per_seq)),
            _arg(slot_mapping, torch.int64, "slot_mapping", dev, (cap,)),
            _arg(positions, i32, "positions", dev, (cap,)),
            _arg(logits_indices, i32, "logits_indices", dev, one), _error(error_word, dev))
    pool.max_tokens = cap


def commit_step(pool: RequestPool, request_ids, q_lens, new_lens=None, error_word=None,
                stream=None, max_tokens=None) -> None:
    """The built step is over: request lengths become ``new_lens`` [S] (None: every new token
    stays, 0: the request is over) and pages behind them return to the pool.  A step that the
    build refused is refused; ``max_tokens`` is what the build had (its slot_mapping's length),
    None for that of the last build with this handle."""
    import torch

    dev, i32 = _pool_device(pool, request_ids), torch.int32
    one = (int(request_ids.shape[0]),)
    cap = getattr(pool, "max_tokens", _capi.MAX_TOKENS) if max_tokens is None else int(max_tokens)
    _sizes(one[0], cap)
    _launch("commit_step", dev, stream, load().mcp_commit_built_step, ctypes.byref(pool),
            _arg(request_ids, i32, "request_ids", dev, one), _arg(q_lens, i32, "q_lens", dev, one),
            _arg(new_lens, i32, "new_lens", dev, one), one[0], cap, _error(error_word, dev))


def _dtype_code(t, name):
    import torch

    dtype = t.dtype
    if dtype is torch.bfloat16:
        return _capi.DTYPE_BF16
    if dtype is torch.float16:
        return _capi.DTYPE_FP16
    if dtype is torch.float32:
        return _capi.DTYPE_FP32
    raise TypeError(f"{name} must be bf16, fp16 or fp32, got {dtype}")


def mixed_conv(x, weight, bias, state, request_ids, cu_seqlens_q, seqlens_k, activation="silu",
               out=None, error_word=None, stream=None):
    """Short causal convolution of every segment of the packed stream, continued from and
    kept in ``state`` (see include/mcp.h): x [T, channels] (rows may be part of wider ones),
    weight [channels, K], bias [channels] or None, state [requests, K - 1, channels], all of
    one type (bf16 or fp16); request_ids, seqlens_k [S], cu_seqlens_q [S + 1] int32.
    ``activation``: "silu" or "none".  Returns ``out`` [T, channels]."""
    import torch

    if activation not in ("silu", "none"):
        raise ValueError("activation must be 'silu' or 'none'")
    dev, dtype, i32 = _gpu(x, "x"), x.dtype, torch.int32
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [T, channels], weight [channels, K], "
                         "state [requests, K - 1, channels]")
    rows = x.shape
    T, d = rows
    K, S, R = weight.shape[1], request_ids.shape[0], state.shape[0]
    _sizes(T, d, K, S, R)
    if out is None:
        out = _empty(rows, dtype, x.device, stream, result=True)
    px, ldx = _row_arg(x, dtype, "x", dev, rows)
    po, ldo = _row_arg(out, dtype, "out", dev, rows)
    desc = _capi.ConvDesc(S, T, R, d, K, _dtype_code(x, "x"), activation == "silu", 0, ldx, ldo)
    _launch("mixed_conv", dev, stream, load().mcp_mixed_conv, ctypes.byref(desc), px,
            _arg(weight, dtype, "weight", dev, (d, K)), _arg(bias, dtype, "bias", dev, (d,)),
            _arg(state, dtype, "state", dev, (R, K - 1, d)),
            _arg(request_ids, i32, "request_ids", dev, (S,)),
            _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, (S,)), po, _error(error_word, dev))
    return out


def mixed_scan(x, dt, A, B, C, state, request_ids, cu_seqlens_q, seqlens_k, D=None, z=None,
               dt_bias=None, softplus=True, out=None, workspace=None, error_word=None,
               stream=None):
    """Selective state space scan of every segment of the packed stream, continued from and
    kept in ``state`` (see include/mcp.h): x, dt and z (or None) [T, channels], B and C
    [T, groups, N] of one type (bf16 or fp16; rows may be part of wider ones); A [channels, N],
    D and dt_bias [channels] (or None) and state [requests, channels, N] fp32; request_ids,
    seqlens_k [S], cu_seqlens_q [S + 1] int32.  ``workspace``: uint8 tensor for long segments
    run in pieces (``mcp_mixed_scan_workspace`` bytes), None to take one from torch for this
    call.  Returns ``out`` [T, channels]."""
    import torch

    dev, dtype = _gpu(x, "x"), x.dtype
    f32, i32 = torch.float32, torch.int32
    if x.dim() != 2 or B.dim() != 3 or state.dim() != 3:
        raise ValueError("x must be [T, channels], B and C [T, groups, N], "
                         "state [requests, channels, N]")
    rows, bc = x.shape, B.shape
    T, d = rows
    G, N, S, R = bc[1], bc[2], request_ids.shape[0], state.shape[0]
    _sizes(T, d, G, N, S, R)
    if out is None:
        out = _empty(rows, dtype, x.device, stream, result=True)
    px, ldx = _row_arg(x, dtype, "x", dev, rows)
    pd, ldd = _row_arg(dt, dtype, "dt", dev, rows)
    pz, ldz = (None, 0) if z is None else _row_arg(z, dtype, "z", dev, rows)
    pb, ldb = _row_arg(B, dtype, "B", dev, (T, G, N))
    pc, ldc = _row_arg(C, dtype, "C", dev, (T, G, N))
    po, ldo = _row_arg(out, dtype, "out", dev, rows)
    desc = _capi.ScanDesc(S, T, R, d, N, G, _dtype_code(x, "x"), bool(softplus), ldx, ldd, ldz,
                          ldb, ldc, ldo)
    tensors = _capi.ScanTensors(
        px, pd, _arg(A, f32, "A", dev, (d, N)), pb, pc, _arg(D, f32, "D", dev, (d,)), pz,
        _arg(dt_bias, f32, "dt_bias", dev, (d,)), _arg(state, f32, "state", dev, (R, d, N)), po)
    if workspace is None and T > S:
        nbytes = ctypes.c_size_t()
        _launch_free("mixed_scan_workspace", dev, load().mcp_mixed_scan_workspace,
                     ctypes.byref(desc), ctypes.byref(nbytes))
        if nbytes.value:
            workspace = _empty(nbytes.value, torch.uint8, x.device, stream)
    _launch("mixed_scan", dev, stream, load().mcp_mixed_scan, ctypes.byref(desc),
            ctypes.byref(tensors), _arg(request_ids, i32, "request_ids", dev, (S,)),
            _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, (S,)),
            _arg(workspace, torch.uint8, "workspace", dev),
            0 if workspace is None else workspace.numel(), _error(error_word, dev))
    return out


def _token_state(seen, counts, vocab_size, dev):
    """Addresses of ``seen`` [R, 2, W] and ``counts`` [R, 32 W], W = ceil(vocab_size / 32)."""
    import torch

    W = (vocab_size + 31) // 32
    if seen.dim() != 3:
        raise ValueError("seen must be [requests, 2, ceil(vocab_size / 32)]")
    R = seen.shape[0]
    return (R, _arg(seen, torch.int32, "seen", dev, (R, 2, W)),
            _arg(counts, torch.int32, "counts", dev, (R, 32 * W)))


def update_token_counts(request_ids, tokens, seen, counts, vocab_size, cu_tokens=None,
                        prompt=False, reset=False, error_word=None, stream=None) -> None:
    """Add tokens to what each request has had (see include/mcp.h): row i's are
    tokens[cu_tokens[i]:cu_tokens[i + 1]] (``cu_tokens`` None: token i alone), added to
    request row request_ids[i] of seen [R, 2, W] and counts [R, 32 W], W = ceil(vocab_size /
    32); all int32 CUDA tensors.  ``prompt``: they are prompt tokens; ``reset``: the rows are
    cleared first."""
    import torch

    dev, i32 = _gpu(request_ids, "request_ids"), torch.int32
    n, rows, V = tokens.shape[0], request_ids.shape[0], int(vocab_size)
    R, ps, pc = _token_state(seen, counts, V, dev)
    _sizes(n, rows, V, R)
    _launch("update_token_counts", dev, stream, load().mcp_update_token_counts,
            _arg(request_ids, i32, "request_ids", dev, (rows,)), rows,
            _arg(tokens, i32, "tokens", dev, (n,)), n,
            _arg(cu_tokens, i32, "cu_tokens", dev, (rows + 1,)), ps, pc, R, V,
            (_capi.COUNT_PROMPT if prompt else 0) | (_capi.COUNT_RESET if reset else 0),
            _error(error_word, dev))


def process_logits(logits, out=None, request_ids=None, seen=None, counts=None, temperature=None,
                   repetition_penalty=None, frequency_penalty=None, presence_penalty=None,
                   bias=None, mask=None, mask_rows=None, error_word=None, stream=None):
    """Biases, penalties for repeated tokens, temperature and grammar masks on logits
    [rows, vocab] (bf16, fp16 or fp32; rows may be part of wider ones), see include/mcp.h.
    ``out``: None for in place, else [rows, vocab] of the logits' type or fp32.  The penalties
    and the temperature are fp32 [rows]; request_ids [rows], seen and counts as in
    ``update_token_counts``; ``bias``: (offsets [rows + 1], tokens, values fp32), the tokens of
    a row strictly increasing; mask [masks, ceil(vocab / 32)] with a 1 bit for every allowed
    token, mask_rows [rows] or None for one mask a row.  Returns the processed logits."""
    import torch

    dev = _gpu(logits, "logits")
    out = logits if out is None else out
    if logits.dim() != 2 or out.shape != logits.shape:
        raise ValueError("logits and out must be [rows, vocab]")
    rows, V = logits.shape
    f32, i32 = torch.float32, torch.int32
    one = (rows,)
    ld = []
    for t, name in ((logits, "logits"), (out, "out")):
        strides = t.stride()
        if V > 1 and strides[1] != 1:
            raise ValueError(f"{name}: a row must be dense, got strides {strides}")
        ld.append(strides[0] if rows > 1 else V)
    if out.get_device() != dev:
        raise ValueError(f"out must be on {logits.device}, got {out.device}")
    R, ps, pc = 0, None, None
    if request_ids is not None:
        if seen is None or counts is None:
            raise ValueError("request_ids needs seen and counts")
        R, ps, pc = _token_state(seen, counts, V, dev)
    off, tok, val, biases = None, None, None, 0
    if bias is not None:
        off, tok, val = bias
        if off is None or tok is None or val is None or tok.dim() != 1:
            raise ValueError("bias must be (offsets [rows + 1], tokens [n], values [n])")
        biases = tok.shape[0]
    masks = 0 if mask is None else mask.shape[0]
    _sizes(rows, V, R, biases, masks)
    desc = _capi.LogitsDesc(rows, V, R, _dtype_code(logits, "logits"), _dtype_code(out, "out"),
                            biases, masks, 0, ld[0], ld[1])
    tensors = _capi.LogitsTensors(
        logits.data_ptr(), out.data_ptr(), _arg(request_ids, i32, "request_ids", dev, one), ps, pc,
        _arg(temperature, f32, "temperature", dev, one),
        _arg(repetition_penalty, f32, "repetition_penalty", dev, one),
        _arg(frequency_penalty, f32, "frequency_penalty", dev, one),
        _arg(presence_penalty, f32, "presence_penalty", dev, one),
        _arg(off, i32, "bias offsets", dev, (rows + 1,)), _arg(tok, i32, "bias tokens", dev),
        _arg(val, f32, "bias values", dev, (biases,)),
        _arg(mask, i32, "mask", dev, (masks, (V + 31) // 32)),
        _arg(mask_rows, i32, "mask_rows", dev, one))
    _launch("process_logits", dev, stream, load().mcp_process_logits, ctypes.byref(desc),
            ctypes.byref(tensors), _error(error_word, dev))
    return out


# ---------------------------------------------------------------------------
# trees of drafted tokens
# ---------------------------------------------------------------------------

def build_tree_masks(parents, cu_seqlens_q, seqlens_k, mask_rows, tree_mask, positions=None,
                     error_word=None, stream=None) -> None:
    """Which tokens of its tree each token of a step sees, and its position (see
    include/mcp.h): parents [T] (the place of a token's parent in its segment, < 0: none),
    cu_seqlens_q [S + 1], seqlens_k [S] and mask_rows [S] (the row of a tree's first token,
    < 0: a causal segment) in; tree_mask [rows, words] and positions [T] (or None) out, all
    int32 CUDA tensors."""
    import torch

    dev, i32 = _gpu(parents, "parents"), torch.int32
    if parents.dim() != 1 or mask_rows.dim() != 1 or tree_mask.dim() != 2:
        raise ValueError("parents must be [T], mask_rows [S], tree_mask [rows, words]")
    T, S = parents.shape[0], mask_rows.shape[0]
    rows, words = tree_mask.shape
    _sizes(T, S, rows, words)
    _launch("build_tree_masks", dev, stream, load().mcp_build_tree_masks,
            _arg(parents, i32, "parents", dev), _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, (S,)), _arg(mask_rows, i32, "mask_rows", dev),
            S, T, rows, words, _arg(tree_mask, i32, "tree_mask", dev),
            _arg(positions, i32, "positions", dev, (T,)), _error(error_word, dev))


def mixed_attn_fwd_tree(plan: Plan, q, k_cache, v_cache, block_tables, cu_seqlens_q, seqlens_k,
                        tree_mask, mask_rows, out, lse=None, workspace=None, stream=None) -> None:
    """``mixed_attn_fwd`` of a step in which segments with mask_rows[s] >= 0 are trees of
    drafted tokens (see include/mcp.h): their tokens see the history, themselves and the tokens
    before them whose bit is set in their row of tree_mask [rows, words] (int32).  The plan is
    made with ``PlanOptions(tree=1)`` and serves any trees of its lengths."""
    import torch

    dev, i32, bf16 = _gpu(q, "q"), torch.int32, torch.bfloat16
    d = plan.desc
    if tree_mask.dim() != 2:
        raise ValueError("tree_mask must be [rows, words]")
    rows, words = tree_mask.shape
    _sizes(rows, words)
    if q.dim() != 3 or q.shape[0] < d.total_q:  # rows behind the step's tokens are padding
        raise ValueError(f"q must be [tokens, H_q, D] with the plan's {d.total_q} tokens")
    heads = (q.shape[0], d.num_q_heads, d.head_dim)
    cache = (d.num_pages, d.page_size, d.num_kv_heads, d.head_dim)
    S = d.num_seqs
    _launch("mixed_attn_fwd_tree", dev, stream, load().mcp_mixed_attn_fwd_tree, ctypes.byref(plan),
            _arg(q, bf16, "q", dev, heads), _arg(k_cache, bf16, "k_cache", dev, cache),
            _arg(v_cache, bf16, "v_cache", dev, cache),
            _arg(block_tables, i32, "block_tables", dev, (S, d.max_pages_per_seq)),
            _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, (S,)), _arg(tree_mask, i32, "tree_mask", dev),
            rows, words, _arg(mask_rows, i32, "mask_rows", dev, (S,)),
            _arg(out, bf16, "out", dev, heads), _arg(lse, torch.float32, "lse", dev, heads[:2]),
            _arg(workspace, torch.uint8, "workspace", dev),
            0 if workspace is None else workspace.numel())


def _prob_rows(t, dtype, name, dev, shape):
    """(address, elements between rows) of [rows, vocab] probabilities."""
    try:
        good = t.dtype is dtype and t.get_device() == dev and t.shape == shape
    except AttributeError:
        good = False
    if not good:
        _refuse(t, dtype, name, dev, shape)
    strides = t.stride()
    if shape[1] > 1 and strides[1] != 1:
        raise ValueError(f"{name}: a row must be dense, got strides {strides}")
    return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1]


def verify_drafts(target_probs, tokens, cu_rows, uniform, final_uniform, parents=None,
                  draft_probs=None, accepted=None, path=None, new_tokens=None, error_word=None,
                  stream=None):
    """Which drafted tokens stay, and the token behind them (see include/mcp.h): target_probs
    [R, vocab] and draft_probs (the same, or None) of one type (bf16, fp16 or fp32; rows may be
    part of wider ones), row i of a segment for what follows its node i; tokens [R], parents [R]
    (None: chains), cu_rows [S + 1] int32; uniform [R] and final_uniform [S] fp32 in [0, 1).
    Returns (accepted [S], path [R], new_tokens [R]), int32: the rows that stay, the root among
    them, their places, and the tokens to go on with, behind them -1."""
    import torch

    dev, dtype = _gpu(target_probs, "target_probs"), target_probs.dtype
    i32, f32 = torch.int32, torch.float32
    if target_probs.dim() != 2 or cu_rows.dim() != 1 or cu_rows.shape[0] == 0:
        raise ValueError("target_probs must be [rows, vocab], cu_rows [segments + 1]")
    shape = target_probs.shape
    R, V = shape
    S = cu_rows.shape[0] - 1
    _sizes(R, V, S)
    pt, ldt = _prob_rows(target_probs, dtype, "target_probs", dev, shape)
    pd, ldd = (None, 0) if draft_probs is None else _prob_rows(draft_probs, dtype, "draft_probs", dev,
                                                               shape)
    device = target_probs.device
    if accepted is None:
        accepted = _empty((S,), i32, device, stream, result=True)
    if path is None:
        path = _empty((R,), i32, device, stream, result=True)
    if new_tokens is None:
        new_tokens = _empty((R,), i32, device, stream, result=True)
    desc = _capi.VerifyDesc(S, R, V, _dtype_code(target_probs, "target_probs"), ldt, ldd)
    tensors = _capi.VerifyTensors(
        pt, pd, _arg(tokens, i32, "tokens", dev, (R,)), _arg(parents, i32, "parents", dev, (R,)),
        _arg(cu_rows, i32, "cu_rows", dev), _arg(uniform, f32, "uniform", dev, (R,)),
        _arg(final_uniform, f32, "final_uniform", dev, (S,)),
        _arg(accepted, i32, "accepted", dev, (S,)), _arg(path, i32, "path", dev, (R,)),
        _arg(new_tokens, i32, "new_tokens", dev, (R,)))
    _launch("verify_drafts", dev, stream, load().mcp_verify_drafts, ctypes.byref(desc),
            ctypes.byref(tensors), _error(error_word, dev))
    return accepted, path, new_tokens


def _layers(caches, name, dev, shape):
    """(shape of one cache, layers, elements between them, array of addresses) of one cache
    [pages, P, H_kv, D], all layers' [layers, pages, P, H_kv, D] (one address), or a list of
    caches (elements 0)."""
    import torch

    bf16 = torch.bfloat16
    if isinstance(caches, torch.Tensor):
        full = caches.shape
        if len(full) == 5:
            one, stride = full[1:], caches.stride(0)
            if full[0] and stride and (shape is None or one == shape):
                # K and V may alternate in one pool: each layer's cache is dense, not all of them
                first = caches if caches.is_contiguous() else caches[0]
                return one, full[0], stride, ctypes.c_void_p(_arg(first, bf16, name, dev))
        elif len(full) == 4:
            caches = (caches,)
        else:
            raise ValueError(f"{name} must be caches [pages, P, H_kv, D] of one or all layers")
    caches = tuple(caches)
    if shape is None and caches:
        _gpu(caches[0], name)
        shape = caches[0].shape
        if len(shape) != 4:
            raise ValueError(f"{name} must be caches [pages, P, H_kv, D]")
    return shape, len(caches), 0, (ctypes.c_void_p * len(caches))(
        *(_arg(c, bf16, name, dev, shape) for c in caches))


def kv_keep_path(k_caches, v_caches, block_tables, cu_seqlens_q, seqlens_k, accepted, path,
                 cu_rows=None, new_lens=None, error_word=None, stream=None):
    """The accepted tokens' K/V moved behind their history, in every layer (see include/mcp.h):
    k_caches, v_caches: lists of bf16 caches [pages, P, H_kv, D], or one tensor [layers, pages, P,
    H_kv, D]; block_tables [S, max_pages_per_seq], cu_seqlens_q [S + 1], seqlens_k [S]; accepted
    [S], path [R] and cu_rows [S + 1] as ``verify_drafts`` takes and gives them (``cu_rows`` None:
    its rows are the step's tokens), all int32 CUDA tensors.  No two caches share memory: one that
    several layers share is given once.  Returns ``new_lens`` [S]: the tokens that each request
    holds now (for ``commit_step``)."""
    import torch

    dev, i32 = _gpu(accepted, "accepted"), torch.int32
    shape, L, stride, ks = _layers(k_caches, "k_caches", dev, None)
    _, more, other, vs = _layers(v_caches, "v_caches", dev, shape)
    if not L or L != more or stride != other:
        raise ValueError("k_caches and v_caches must have the same layers, one at least, both listed "
                         "or both one tensor")
    if accepted.dim() != 1 or path.dim() != 1 or block_tables.dim() != 2:
        raise ValueError("accepted must be [S], path [R], block_tables [S, max_pages_per_seq]")
    S, R = accepted.shape[0], path.shape[0]
    pages, P, H, D = shape
    width = block_tables.shape[1]
    _sizes(S, R, L, pages, P, H, D, width)
    one = (S,)
    if new_lens is None:
        new_lens = _empty(one, i32, accepted.device, stream, result=True)
    desc = _capi.KeepDesc(S, R, L, H, D, P, width, pages, stride)
    _launch("kv_keep_path", dev, stream, load().mcp_kv_keep_path, ctypes.byref(desc),
            ctypes.byref(ks), ctypes.byref(vs), _arg(block_tables, i32, "block_tables", dev, (S, width)),
            _arg(cu_seqlens_q, i32, "cu_seqlens_q", dev, (S + 1,)),
            _arg(seqlens_k, i32, "seqlens_k", dev, one), _arg(cu_rows, i32, "cu_rows", dev, (S + 1,)),
            _arg(accepted, i32, "accepted", dev, one), _arg(path, i32, "path", dev),
            _arg(new_lens, i32, "new_lens", dev, one), _error(error_word, dev))
    return new_lens
