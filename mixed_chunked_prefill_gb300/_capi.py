"""ctypes view of the C ABI declared in include/mcp.h (argument marshalling only)."""

from __future__ import annotations

import ctypes
import os
import warnings
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libmcp.so")

MCP_OK = 0
MCP_ERR_INVALID_ARG = 1
MCP_ERR_UNSUPPORTED = 2
MCP_ERR_WORKSPACE_TOO_SMALL = 3
MCP_ERR_CUDA = 4
MCP_ERR_TIMEOUT = 5
MCP_ERR_DEVICE_CHECK = 6

DEVERR_TIMEOUT = 0x1
DEVERR_PAGE_RANGE = 0x2
DEVERR_SLOT_RANGE = 0x4
DEVERR_ROW_RANGE = 0x8
DEVERR_ITEM_KIND = 0x10
DEVERR_SLOT_DUP = 0x20
DEVERR_NO_PAGES = 0x40
DEVERR_REQUEST = 0x80
DEVERR_TOKEN_RANGE = 0x100
DEVERR_SEGMENT = 0x200
DEVERR_TREE = 0x400
DEVERR_PROBS = 0x800
BUILD_CHECKED = 0x1
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
COUNT_PROMPT = 0x1
COUNT_RESET = 0x2
MAX_TOKENS = 1 << 30  # of a build of step tables
MAX_MASK_WORDS = 32  # of a tree's mask row


class AttnDesc(ctypes.Structure):
    _fields_ = [
        ("num_seqs", c_int32),
        ("total_q", c_int32),
        ("num_q_heads", c_int32),
        ("num_kv_heads", c_int32),
        ("head_dim", c_int32),
        ("page_size", c_int32),
        ("max_pages_per_seq", c_int32),
        ("num_pages", c_int32),
        ("sm_scale", c_float),
    ]


class PlanOptions(ctypes.Structure):
    """``mcp_plan_options``.  A name that is none of its fields would only become an attribute of
    the Python object, which the planner never sees: it warns."""

    _fields_ = [
        ("num_sms", c_int32),
        ("decode_split_tokens", c_int32),
        ("prefill_split_tokens", c_int32),
        ("test_stall", c_int32),
        ("tree", c_int32),
        ("reserved", c_int32 * 3),
    ]

    def __setattr__(self, name, value):
        names = [n for n, _ in self._fields_]
        if name not in names:
            warnings.warn(f"PlanOptions has no option {name!r}, which changes nothing (it has "
                          f"{', '.join(names)})", stacklevel=2)
        super().__setattr__(name, value)


class Plan(ctypes.Structure):
    _fields_ = [
        ("magic", c_int32),
        ("num_items", c_int32),
        ("num_decode_items", c_int32),
        ("num_prefill_items", c_int32),
        ("num_combine", c_int32),
        ("decode_split_tokens", c_int32),
        ("prefill_split_tokens", c_int32),
        ("num_sms", c_int32),
        ("partial_rows", c_int64),
        ("off_items", c_int64),
        ("off_combine", c_int64),
        ("off_part_o", c_int64),
        ("off_part_lse", c_int64),
        ("off_error", c_int64),
        ("workspace_bytes", c_int64),
        ("desc", AttnDesc),
        ("combine_rows", c_int32),
        ("test_stall", c_int32),
        ("tree", c_int32),
        ("reserved", c_int32 * 5),
    ]


class SchedConfig(ctypes.Structure):
    _fields_ = [
        ("max_num_batched_tokens", c_int32),
        ("long_prefill_token_threshold", c_int32),
        ("max_num_seqs", c_int32),
        ("num_pages", c_int32),
        ("page_size", c_int32),
        ("max_pages_per_seq", c_int32),
        ("preempt_swap", c_int32),
        ("num_host_pages", c_int32),
        ("reserved", c_int32 * 4),
    ]


class SchedOutput(ctypes.Structure):
    _fields_ = [
        ("num_seqs", c_int32),
        ("total_q", c_int32),
        ("request_ids", POINTER(c_int64)),
        ("cu_seqlens_q", POINTER(c_int32)),
        ("seqlens_k", POINTER(c_int32)),
        ("block_tables", POINTER(c_int32)),
        ("sample_mask", POINTER(ctypes.c_uint8)),
        ("logits_indices", POINTER(c_int32)),
        ("num_logits", c_int32),
        ("num_swap_out", c_int32),
        ("swap_out_device_pages", POINTER(c_int32)),
        ("swap_out_host_pages", POINTER(c_int32)),
        ("num_swap_in", c_int32),
        ("swap_in_host_pages", POINTER(c_int32)),
        ("swap_in_device_pages", POINTER(c_int32)),
        ("num_preempted", c_int32),
        ("preempted_ids", POINTER(c_int64)),
        ("reserved", c_int32 * 4),
    ]


class HostStepLimits(ctypes.Structure):
    _fields_ = [
        ("max_tokens", c_int32),
        ("max_seqs", c_int32),
        ("max_pages_per_seq", c_int32),
        ("reserved0", c_int32),
        ("workspace_bytes", c_int64),
        ("list_bytes", c_int64),
        ("reserved", c_int32 * 4),
    ]


class RequestPool(ctypes.Structure):
    _fields_ = [
        ("max_requests", c_int32),
        ("max_pages_per_seq", c_int32),
        ("page_size", c_int32),
        ("num_pages", c_int32),
        ("request_pages", c_void_p),
        ("request_lens", c_void_p),
        ("free_pages", c_void_p),
        ("free_count", c_void_p),
    ]


class ConvDesc(ctypes.Structure):
    _fields_ = [
        ("num_seqs", c_int32),
        ("total_tokens", c_int32),
        ("num_requests", c_int32),
        ("channels", c_int32),
        ("width", c_int32),
        ("dtype", c_int32),
        ("activation", c_int32),
        ("reserved", c_int32),
        ("x_stride", c_int64),
        ("out_stride", c_int64),
    ]


class ScanDesc(ctypes.Structure):
    _fields_ = [
        ("num_seqs", c_int32),
        ("total_tokens", c_int32),
        ("num_requests", c_int32),
        ("channels", c_int32),
        ("state_size", c_int32),
        ("num_groups", c_int32),
        ("dtype", c_int32),
        ("softplus", c_int32),
        ("x_stride", c_int64),
        ("dt_stride", c_int64),
        ("z_stride", c_int64),
        ("b_stride", c_int64),
        ("c_stride", c_int64),
        ("out_stride", c_int64),
    ]


class ScanTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state",
                                        "out")]


class LogitsDesc(ctypes.Structure):
    _fields_ = [
        ("num_rows", c_int32),
        ("vocab_size", c_int32),
        ("num_requests", c_int32),
        ("dtype", c_int32),
        ("out_dtype", c_int32),
        ("num_biases", c_int32),
        ("num_masks", c_int32),
        ("reserved", c_int32),
        ("logits_stride", c_int64),
        ("out_stride", c_int64),
    ]


class LogitsTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in (
        "logits", "out", "request_ids", "seen", "counts", "temperature", "repetition_penalty",
        "frequency_penalty", "presence_penalty", "bias_offsets", "bias_tokens", "bias_values",
        "mask", "mask_rows")]


class VerifyDesc(ctypes.Structure):
    _fields_ = [
        ("num_seqs", c_int32),
        ("total_rows", c_int32),
        ("vocab_size", c_int32),
        ("dtype", c_int32),
        ("target_stride", c_int64),
        ("draft_stride", c_int64),
    ]


class VerifyTensors(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in (
        "target", "draft", "tokens", "parents", "cu_rows", "uniform", "final_uniform", "accepted",
        "path", "new_tokens")]


class KeepDesc(ctypes.Structure):
    _fields_ = [(n, c_int32) for n in (
        "num_seqs", "total_rows", "num_layers", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pages")] + [("layer_stride", c_int64)]


# name -> (restype, argtypes); every symbol include/mcp.h declares
SIGNATURES = {
    "mcp_status_string": (c_char_p, [c_int32]),
    "mcp_last_error": (c_char_p, []),
    "mcp_abi_version": (c_int32, []),
    "mcp_build_flags": (c_int32, []),
    "mcp_paged_kv_append": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32,
                                      c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "mcp_build_slot_mapping": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p,
                                         c_void_p, c_void_p]),
    "mcp_mixed_attn_plan": (c_int32, [POINTER(AttnDesc), c_void_p, c_void_p, POINTER(PlanOptions),
                                      POINTER(Plan), c_void_p, c_size_t, c_void_p]),
    "mcp_mixed_attn_plan_host": (c_int32, [POINTER(AttnDesc), c_void_p, c_void_p,
                                           POINTER(PlanOptions), POINTER(Plan), c_void_p,
                                           c_size_t]),
    "mcp_mixed_attn_fwd": (c_int32, [POINTER(Plan), c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                     c_void_p]),
    "mcp_mixed_attn_fwd_noalloc": (c_int32, [POINTER(AttnDesc), c_void_p, c_void_p,
                                             POINTER(PlanOptions), c_void_p, c_void_p, c_void_p,
                                             c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                             c_void_p, c_void_p]),
    "mcp_mixed_attn_fwd_varlen": (c_int32, [POINTER(Plan), c_void_p, c_void_p, c_void_p,
                                            c_void_p, c_void_p, c_int64, c_void_p, c_void_p,
                                            c_void_p, c_size_t, c_void_p]),
    "mcp_check_device_errors": (c_int32, [c_void_p, c_void_p]),
    "mcp_workspace_error_word": (c_void_p, [POINTER(Plan), c_void_p]),
    "mcp_merge_states": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32,
                                   c_void_p, c_void_p, c_void_p]),
    "mcp_build_logits_indices": (c_int32, [c_int32, c_void_p, c_void_p, c_void_p,
                                           POINTER(c_int32)]),
    "mcp_mixed_attn_plan_rows": (c_int32, [POINTER(AttnDesc), c_void_p, c_void_p, c_void_p,
                                           c_int32, POINTER(PlanOptions), POINTER(Plan),
                                           c_void_p, c_size_t, c_void_p]),
    "mcp_mixed_attn_plan_rows_host": (c_int32, [POINTER(AttnDesc), c_void_p, c_void_p,
                                                c_void_p, c_int32, POINTER(PlanOptions),
                                                POINTER(Plan), c_void_p, c_size_t]),
    "mcp_kv_copy_pages": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                                    c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "mcp_gather_rows": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p,
                                  c_void_p, c_void_p]),
    "mcp_sched_create": (c_int32, [POINTER(SchedConfig), POINTER(c_void_p)]),
    "mcp_sched_add_request": (c_int32, [c_void_p, c_int64, c_int32, c_int32, c_int32]),
    "mcp_sched_schedule": (c_int32, [c_void_p, POINTER(SchedOutput)]),
    "mcp_sched_finish_step": (c_int32, [c_void_p, POINTER(c_int32), c_void_p]),
    "mcp_sched_stats": (c_int32, [c_void_p, POINTER(c_int32), POINTER(c_int32), POINTER(c_int32),
                                  POINTER(c_int64), POINTER(c_int32)]),
    "mcp_sched_destroy": (c_int32, [c_void_p]),
    "mcp_host_step_arena_bytes": (c_int32, [POINTER(AttnDesc), POINTER(HostStepLimits),
                                            POINTER(c_size_t), POINTER(c_size_t)]),
    "mcp_host_step_create": (c_int32, [POINTER(AttnDesc), POINTER(HostStepLimits), c_void_p,
                                       c_size_t, c_void_p, c_size_t, c_void_p,
                                       POINTER(c_void_p)]),
    "mcp_host_step_run": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    POINTER(c_int64)]),
    "mcp_host_step_wait": (c_int32, [c_void_p, c_int64]),
    "mcp_host_step_destroy": (c_int32, [c_void_p]),
    "mcp_build_step_tables": (c_int32, [POINTER(RequestPool), c_void_p, c_void_p, c_int32, c_int32,
                                        c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_void_p]),
    "mcp_commit_built_step": (c_int32, [POINTER(RequestPool), c_void_p, c_void_p, c_void_p, c_int32,
                                        c_int32, c_void_p, c_void_p]),
    "mcp_commit_step": (c_int32, [POINTER(RequestPool), c_void_p, c_void_p, c_void_p, c_int32,
                                  c_void_p, c_void_p]),
    "mcp_mixed_conv": (c_int32, [POINTER(ConvDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "mcp_mixed_scan": (c_int32, [POINTER(ScanDesc), POINTER(ScanTensors), c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "mcp_mixed_scan_workspace": (c_int32, [POINTER(ScanDesc), POINTER(c_size_t)]),
    "mcp_update_token_counts": (c_int32, [c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                          c_void_p, c_int32, c_int32, c_int32, c_void_p,
                                          c_void_p]),
    "mcp_process_logits": (c_int32, [POINTER(LogitsDesc), POINTER(LogitsTensors), c_void_p,
                                     c_void_p]),
    "mcp_build_tree_masks": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                       c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "mcp_mixed_attn_fwd_tree": (c_int32, [POINTER(Plan), c_void_p, c_void_p, c_void_p, c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                          c_void_p]),
    "mcp_verify_drafts": (c_int32, [POINTER(VerifyDesc), POINTER(VerifyTensors), c_void_p,
                                    c_void_p]),
    "mcp_kv_keep_path": (c_int32, [POINTER(KeepDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p]),
}

_lib = None


def open_library(path: str):
    """A ctypes handle on the library at ``path`` with every signature set."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(the CUDA library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load(path: str = LIB_PATH):
    """Load the CUDA library; raise if it was not built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = open_library(path)
    return _lib


class MCPError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        self.status = status
        msg = lib.mcp_last_error().decode(errors="replace")
        name = lib.mcp_status_string(status).decode()
        super().__init__(f"{where}: {name}: {msg}")


def check(status: int, where: str) -> None:
    if status != MCP_OK:
        raise MCPError(status, where)
