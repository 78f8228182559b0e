"""Step runners over the C ABI: the calls one layer of a chunked-prefill
serving step makes ([W] wangyu.me "大语言模型推理优化（二）：Chunked Prefill",
section "输入组装": write the new K/V through slot_mapping, then run the varlen
paged attention).

``MixedStep`` keeps one step's metadata, plan and workspace on the device and
runs append + attention on device tensors.  ``HostStep`` is the end-to-end
path from host buffers over the library's pipelined host step: each call
copies the step's inputs and metadata to the device, plans on the host,
appends, attends and copies the output back, with up to two steps in flight
(the copies of one step overlap the kernels of the other).
"""

from __future__ import annotations

import numpy as np

from . import (
    _capi,
    PlanOptions,
    build_slot_mapping,
    build_step_tables,
    build_tree_masks,
    check_device_errors,
    commit_step,
    kv_keep_path,
    make_desc,
    make_request_pool,
    mixed_attn_fwd,
    mixed_attn_fwd_tree,
    mixed_attn_plan,
    mixed_attn_plan_rows,
    paged_kv_append,
    process_logits,
    update_token_counts,
    workspace_error_word,
)


def _i32(a):
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _i64(a):
    return np.asarray(a, dtype=np.int64)


def _on_stream(stream, device):
    """Allocations and copies inside belong to ``stream`` of ``device`` (None: the current one)."""
    import contextlib

    import torch

    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                             else torch.cuda.ExternalStream(int(stream), device))


class StepTrees:
    """Trees of drafted tokens of one step: their visibility masks, and the positions of all
    of the step's tokens (``mcp_build_tree_masks``).  ``trees``: which segments are trees
    (the others are causal: chunks, decodes); ``parents`` [T]: for each token of the step the
    place of its parent in its segment, < 0: none (not looked at in causal segments)."""

    def __init__(self, cu_seqlens_q, cu_d, seqlens_k_d, trees, parents, error_word=None,
                 stream=None):
        import torch

        cu, dev = _i64(cu_seqlens_q), cu_d.device
        q = np.diff(cu)
        is_tree = np.asarray(trees, dtype=bool)
        if is_tree.shape != q.shape:
            raise ValueError("trees must be one truth value a segment")
        sizes = np.where(is_tree, q, 0)
        rows = np.concatenate([[0], np.cumsum(sizes)])
        words = max(1, -(-int(sizes.max(initial=0)) // 32))
        if words > _capi.MAX_MASK_WORDS:
            raise ValueError(f"a tree of {int(sizes.max())} tokens > {32 * _capi.MAX_MASK_WORDS}")
        with _on_stream(stream, dev):
            if not isinstance(parents, torch.Tensor):
                parents = torch.from_numpy(_i32(parents))
            self.parents = parents.to(device=dev, dtype=torch.int32)
            self.mask_rows = torch.from_numpy(_i32(np.where(is_tree, rows[:-1], -1))).to(dev)
            self.tree_mask = torch.zeros((int(rows[-1]), words), dtype=torch.int32, device=dev)
            if self.parents.dim() != 1 or self.parents.shape[0] < int(cu[-1]):
                raise ValueError("parents must be [T], an entry for each token of the step")
            self.positions = torch.zeros(self.parents.shape[0], dtype=torch.int32, device=dev)
            build_tree_masks(self.parents, cu_d, seqlens_k_d, self.mask_rows, self.tree_mask,
                             self.positions, error_word, stream)


class MixedStep:
    """Device-side state of one step: metadata, slot mapping, plan, workspace."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale,
                 cu_seqlens_q, seqlens_k, block_tables, device="cuda", options=None,
                 stream=None, rows=None, trees=None, parents=None):
        """``rows``: None for every query row, else the token indices (e.g.
        logits_indices) whose attention rows this step computes.  ``trees``, ``parents``:
        None, or the step's trees of drafted tokens (see ``StepTrees``, kept as ``trees``)."""
        import torch

        self.cu_h = _i32(cu_seqlens_q)
        self.sk_h = _i32(seqlens_k)
        self.bt_h = _i32(block_tables)
        if self.bt_h.ndim != 2:
            raise ValueError("block_tables must be [num_seqs, max_pages_per_seq]")
        S = len(self.sk_h)
        self.desc = make_desc(S, int(self.cu_h[-1]), num_q_heads, num_kv_heads, head_dim,
                              page_size, self.bt_h.shape[1], num_pages, sm_scale)
        self.options = options
        self.stream = stream
        self.device = device
        self.slots_h = build_slot_mapping(self.bt_h, self.cu_h, self.sk_h, page_size, num_pages)
        self.cu_d = torch.from_numpy(self.cu_h).to(device)
        self.sk_d = torch.from_numpy(self.sk_h).to(device)
        self.bt_d = torch.from_numpy(self.bt_h).to(device)
        self.slots_d = torch.from_numpy(self.slots_h).to(device)
        self._plan(rows, trees, parents)

    @classmethod
    def from_tables(cls, tables, num_q_heads, num_kv_heads, head_dim, sm_scale, options=None,
                    stream=None, rows=None, trees=None, parents=None):
        """A step whose tables and slots were built on the device (``RequestTables.step``):
        nothing but the work lists is copied to the device.  Where they are padded
        (``max_tokens``), ``append`` takes the step's tokens alone or padded ones as well."""
        self = cls.__new__(cls)
        pool = tables.pool
        self.cu_h, self.sk_h = tables.cu_h, tables.sk_h
        self.desc = make_desc(len(self.sk_h), int(self.cu_h[-1]), num_q_heads, num_kv_heads,
                              head_dim, pool.page_size, pool.max_pages_per_seq, pool.num_pages,
                              sm_scale)
        self.options, self.stream, self.device = options, stream, tables.block_tables.device
        self.tables = tables
        self.cu_d, self.sk_d = tables.cu_seqlens_q, tables.seqlens_k
        self.bt_d, self.slots_d = tables.block_tables, tables.slot_mapping
        self._plan(rows, trees, parents)
        return self

    def _plan(self, rows, trees=None, parents=None):
        import torch

        options, device, stream = self.options, self.device, self.stream
        self.trees = None
        if (trees is None) != (parents is None):
            raise ValueError("trees and parents go together")
        if trees is not None:
            options = PlanOptions.from_buffer_copy(options) if options is not None else PlanOptions()
            options.tree = 1
        if rows is None:
            def planner(ws=None, st=None):
                return mixed_attn_plan(self.desc, self.cu_h, self.sk_h, options, ws, st)
        else:
            self.rows_h = _i32(rows)

            def planner(ws=None, st=None):
                return mixed_attn_plan_rows(self.desc, self.cu_h, self.sk_h, self.rows_h,
                                            options, ws, st)
        sizing = planner()
        self.workspace = torch.empty(max(256, int(sizing.workspace_bytes)), dtype=torch.uint8,
                                     device=device)
        self.plan = planner(self.workspace, stream)
        self.error_word = workspace_error_word(self.plan, self.workspace)
        if trees is not None:
            self.trees = StepTrees(self.cu_h, self.cu_d, self.sk_d, trees, parents,
                                   self.error_word, stream)

    def append(self, k_new, v_new, k_cache, v_cache):
        slots, n = self.slots_d, int(k_new.shape[0])
        if int(self.cu_h[-1]) <= n < len(slots):  # a padded slot map (from_tables)
            slots = slots[:n]
        paged_kv_append(k_new, v_new, slots, k_cache, v_cache, self.error_word, self.stream)

    def attention(self, q, k_cache, v_cache, out, lse=None):
        if self.trees is not None:
            mixed_attn_fwd_tree(self.plan, q, k_cache, v_cache, self.bt_d, self.cu_d, self.sk_d,
                                self.trees.tree_mask, self.trees.mask_rows, out, lse,
                                self.workspace, self.stream)
            return
        mixed_attn_fwd(self.plan, q, k_cache, v_cache, self.bt_d, self.cu_d, self.sk_d, out, lse,
                       self.workspace, self.stream)

    def run(self, q, k_new, v_new, k_cache, v_cache, out, lse=None):
        self.append(k_new, v_new, k_cache, v_cache)
        self.attention(q, k_cache, v_cache, out, lse)

    def keep(self, k_caches, v_caches, accepted, path, cu_rows=None):
        """Move the accepted paths (``verify_drafts``) behind their histories in all layers'
        caches; returns the tokens that each request holds then (``RequestTables.commit``)."""
        return kv_keep_path(k_caches, v_caches, self.bt_d, self.cu_d, self.sk_d, accepted, path,
                            cu_rows, None, self.error_word, self.stream)

    def check(self):
        """Synchronise and raise if a device-side check or bounded wait failed."""
        check_device_errors(self.error_word, self.stream)


class StepTables:
    """One step of ``RequestTables``: its metadata on the device (and the lengths on the
    host), valid until the next commit of the same tables, which may be this step's only."""

    def __init__(self, tables, request_ids, q_lens, max_tokens, stream):
        import torch

        self.pool, self.after = tables.pool, tables.commits
        dev = tables.device
        ids, q = _i64(request_ids), _i64(q_lens)  # checked before they become 32 bits
        if ids.ndim != 1 or ids.shape != q.shape:
            raise ValueError("request_ids and q_lens must be [num_seqs]")
        live = ids >= 0
        if (ids >= self.pool.max_requests).any() or len(set(ids[live])) != int(live.sum()):
            raise ValueError("request_ids must be distinct rows of the pool (or < 0)")
        if (q < 0).any():
            raise ValueError("q_lens must be >= 0")
        q = np.where(live, q, 0)
        had = np.where(live, tables.lens_h[np.where(live, ids, 0)], 0)
        P = self.pool.page_size
        if (q > self.pool.max_pages_per_seq * P - had).any():
            raise ValueError("a request needs more than max_pages_per_seq pages")
        self.new_pages = int((-(-(had + q) // P) - -(-had // P)).sum())
        if self.new_pages > tables.free_h:
            raise ValueError(f"{self.new_pages} new pages, {tables.free_h} are free")
        S, T = len(ids), int(q.sum())
        cap = T if max_tokens is None else int(max_tokens)
        if T > min(cap, _capi.MAX_TOKENS):
            raise ValueError(f"{T} tokens > max_tokens {min(cap, _capi.MAX_TOKENS)}")
        ids, q, self.sk_h = _i32(np.maximum(ids, -1 << 31)), _i32(q), _i32(had + q)
        self.ids_h, self.q_h = ids, q
        self.cu_h = _i32(np.concatenate([[0], np.cumsum(q)]))
        with _on_stream(stream, dev):
            both = torch.from_numpy(np.concatenate([ids, q])).to(dev)
            self.request_ids, self.q_lens = both[:S], both[S:]
            i32 = dict(dtype=torch.int32, device=dev)
            self.cu_seqlens_q = torch.empty(S + 1, **i32)
            self.seqlens_k = torch.empty(S, **i32)
            self.block_tables = torch.empty((S, self.pool.max_pages_per_seq), **i32)
            self.slot_mapping = torch.empty(cap, dtype=torch.int64, device=dev)
            self.positions = torch.empty(cap, **i32)
            self.logits_indices = torch.empty(S, **i32)
            self._build(tables, stream)

    def _build(self, tables, stream):
        build_step_tables(self.pool, self.request_ids, self.q_lens, self.cu_seqlens_q,
                          self.seqlens_k, self.block_tables, self.slot_mapping, self.positions,
                          self.logits_indices, tables.error_word, stream)
        tables.last = self


class RequestTables:
    """Page tables, lengths and free pages of all requests on the device
    (``mcp_build_step_tables`` / ``mcp_commit_step``), with the lengths mirrored on the host
    for the planner.  ``step`` builds one step's tables from request rows and their new
    tokens, ``commit`` moves the requests on, ``release`` ends requests.  One stream."""

    def __init__(self, num_pages, page_size, max_requests, max_pages_per_seq, device="cuda"):
        import torch

        i32 = dict(dtype=torch.int32, device=device)
        self.request_pages = torch.full((max_requests, max_pages_per_seq), -1, **i32)
        self.request_lens = torch.zeros(max_requests, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        self.error_word = torch.zeros(1, **i32)
        self.device = self.request_pages.device
        self.pool = make_request_pool(self.request_pages, self.request_lens, self.free_pages,
                                      self.free_count, page_size)
        self.lens_h = np.zeros(max_requests, dtype=np.int64)
        self.free_h = int(num_pages)
        self.commits = 0
        self.last = None  # the step built last: the page rows hold its new pages

    def step(self, request_ids, q_lens, max_tokens=None, stream=None) -> StepTables:
        """Tables of a step in which request row request_ids[s] runs q_lens[s] new tokens
        (request_ids[s] < 0: a padding segment).  ``max_tokens``: length of slot_mapping and
        positions (padded behind the step's tokens), default the step's tokens."""
        return StepTables(self, request_ids, q_lens, max_tokens, stream)

    def commit(self, step: StepTables, new_lens=None, stream=None) -> None:
        """The step ran: its requests hold their new tokens, or new_lens[s] tokens (fewer
        after rejected speculated tokens, 0: the request is over)."""
        import torch

        if step.pool is not self.pool or step.after != self.commits:
            raise ValueError("the step was built before another commit, or from other tables")
        live = step.ids_h >= 0
        after = step.sk_h if new_lens is None else _i64(new_lens)
        if after.shape != step.sk_h.shape or ((after < 0) | (after > step.sk_h))[live].any():
            raise ValueError("new_lens must be [num_seqs], at most the step's lengths")
        with _on_stream(stream, self.device):
            if step is not self.last:  # another step entered its pages since: the same again
                step._build(self, stream)
            to = None if new_lens is None else torch.from_numpy(_i32(after)).to(self.device)
            commit_step(self.pool, step.request_ids, step.q_lens, to, self.error_word, stream,
                        max_tokens=step.slot_mapping.shape[0])
        self.commits += 1
        self.last = None
        P = self.pool.page_size
        kept = -(-after // P) - -(-step.sk_h // P)
        self.lens_h[step.ids_h[live]] = after[live]
        self.free_h -= step.new_pages + int(kept[live].sum())

    def release(self, request_ids, stream=None) -> None:
        """End requests: their pages are free and their rows may be used again."""
        ids = _i64(request_ids)
        none = np.zeros(len(ids), dtype=np.int32)
        self.commit(self.step(ids, none, stream=stream), none, stream)

    def check(self, stream=None) -> None:
        """Synchronise and raise if a step was refused on the device."""
        check_device_errors(self.error_word.data_ptr(), stream)


class LogitsState:
    """Which tokens each request has had, on the device, for the penalties of
    ``process_logits``: rows are the request rows of the step."""

    def __init__(self, max_requests, vocab_size, device="cuda"):
        import torch

        words = -(-vocab_size // 32)
        self.vocab_size = int(vocab_size)
        self.seen = torch.zeros((max_requests, 2, words), dtype=torch.int32, device=device)
        self.counts = torch.zeros((max_requests, 32 * words), dtype=torch.int32, device=device)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)

    def admit(self, request_ids, tokens, cu_tokens, stream=None) -> None:
        """New requests take rows: the rows are cleared and their prompts' tokens marked."""
        update_token_counts(request_ids, tokens, self.seen, self.counts, self.vocab_size,
                            cu_tokens, prompt=True, reset=True, error_word=self.error_word,
                            stream=stream)

    def add(self, request_ids, tokens, cu_tokens=None, stream=None) -> None:
        """Sampled tokens: one a row, or tokens[cu_tokens[i]:cu_tokens[i + 1]]."""
        update_token_counts(request_ids, tokens, self.seen, self.counts, self.vocab_size,
                            cu_tokens, error_word=self.error_word, stream=stream)

    def process(self, logits, request_ids, out=None, stream=None, **kw):
        """``process_logits`` with this state (temperature, penalties, bias, mask by name)."""
        return process_logits(logits, out, request_ids, self.seen, self.counts,
                              error_word=self.error_word, stream=stream, **kw)

    def check(self, stream=None) -> None:
        """Synchronise and raise if a row or token was out of range."""
        check_device_errors(self.error_word.data_ptr(), stream)


def write_history(block_tables, hist_lens, k_hist, v_hist, k_cache, v_cache, page_size,
                  stream=None):
    """Fill positions 0..hist_lens[s]-1 of every sequence from packed k_hist /
    v_hist [sum(hist_lens), H_kv, D] (device bf16), through the same slot
    mapping and append kernel a step uses."""
    import torch

    hist = _i32(hist_lens)
    cu = np.concatenate([[0], np.cumsum(hist)]).astype(np.int32)
    if int(cu[-1]) == 0:
        return
    slots = build_slot_mapping(block_tables, cu, hist, page_size, int(k_cache.shape[0]))
    paged_kv_append(k_hist, v_hist, torch.from_numpy(slots).to(k_cache.device), k_cache, v_cache,
                    stream=stream)


class HostStep:
    """End-to-end steps from host memory (``mcp_host_step_*``).

    ``run`` enqueues one step and returns its ticket without waiting: the
    copy-in of q, k_new, v_new (page-locked host tensors, left unchanged until
    the step is waited for), host planning, append, attention and the
    copy-out into ``out_h`` (and ``lse_h``).  ``wait(ticket)`` blocks until
    that step's outputs are in host memory and raises on a device-side error.
    Calling the object runs one step and waits for it.  The device and
    page-locked arenas are torch tensors owned by this object; the KV cache
    is the caller's device state.
    """

    def __init__(self, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale,
                 max_tokens, max_seqs, max_pages_per_seq, device="cuda", stream=None,
                 workspace_bytes=0, list_bytes=0):
        import ctypes

        import torch

        from . import _capi, load

        self._lib = load()
        self.hq, self.hkv, self.D, self.P = num_q_heads, num_kv_heads, head_dim, page_size
        self.mp = int(max_pages_per_seq)
        self.stream = stream if stream is not None else torch.cuda.current_stream(device)
        shape = make_desc(0, 0, num_q_heads, num_kv_heads, head_dim, page_size, 1, num_pages,
                          sm_scale)
        lim = _capi.HostStepLimits(int(max_tokens), int(max_seqs), self.mp, 0,
                                   int(workspace_bytes), int(list_bytes), (ctypes.c_int32 * 4)())
        dbytes, hbytes = ctypes.c_size_t(), ctypes.c_size_t()
        _capi.check(self._lib.mcp_host_step_arena_bytes(ctypes.byref(shape), ctypes.byref(lim),
                                                        ctypes.byref(dbytes), ctypes.byref(hbytes)),
                    "host_step_arena_bytes")
        # arenas: torch's device and page-locked allocations are 256-byte aligned
        self.device_arena = torch.empty(dbytes.value, dtype=torch.uint8, device=device)
        self.host_arena = torch.empty(hbytes.value, dtype=torch.uint8, pin_memory=True)
        handle = ctypes.c_void_p()
        _capi.check(self._lib.mcp_host_step_create(
            ctypes.byref(shape), ctypes.byref(lim), ctypes.c_void_p(self.device_arena.data_ptr()),
            dbytes.value, ctypes.c_void_p(self.host_arena.data_ptr()), hbytes.value,
            ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(handle)), "host_step_create")
        self._h = handle
        self._keep = {}  # host arrays a ticket's copies still read / write
        self.h2d_bytes = 0
        self.d2h_bytes = 0

    def run(self, q_h, k_new_h, v_new_h, cu_seqlens_q, seqlens_k, block_tables, k_cache,
            v_cache, out_h, lse_h=None) -> int:
        import ctypes

        import torch

        from . import _capi

        cu = _i32(cu_seqlens_q)
        sk = _i32(seqlens_k)
        bt = _i32(block_tables)
        S = len(sk)
        if bt.ndim != 2 or bt.shape[0] != S or bt.shape[1] > self.mp:
            raise ValueError(f"block_tables must be [S, <= {self.mp}]")
        if bt.shape[1] < self.mp:
            full = np.full((S, self.mp), -1, dtype=np.int32)
            full[:, :bt.shape[1]] = bt
            bt = full
        T = int(cu[-1]) if len(cu) else 0
        for t, name, dt in ((q_h, "q", torch.bfloat16), (k_new_h, "k_new", torch.bfloat16),
                            (v_new_h, "v_new", torch.bfloat16), (out_h, "out", torch.bfloat16)):
            if t.is_cuda or t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous host {dt} tensor")
        if lse_h is not None and (lse_h.is_cuda or lse_h.dtype != torch.float32):
            raise ValueError("lse must be a host float32 tensor")
        if q_h.numel() < T * self.hq * self.D or out_h.numel() < T * self.hq * self.D:
            raise ValueError("q / out smaller than [T, H_q, D]")
        if k_new_h.numel() < T * self.hkv * self.D or v_new_h.numel() < T * self.hkv * self.D:
            raise ValueError("k_new / v_new smaller than [T, H_kv, D]")
        ticket = ctypes.c_int64(-1)
        st = self._lib.mcp_host_step_run(
            self._h, S, cu.ctypes.data_as(ctypes.c_void_p), sk.ctypes.data_as(ctypes.c_void_p),
            bt.ctypes.data_as(ctypes.c_void_p), ctypes.c_void_p(q_h.data_ptr()),
            ctypes.c_void_p(k_new_h.data_ptr()), ctypes.c_void_p(v_new_h.data_ptr()),
            ctypes.c_void_p(k_cache.data_ptr()), ctypes.c_void_p(v_cache.data_ptr()),
            ctypes.c_void_p(out_h.data_ptr()),
            ctypes.c_void_p(lse_h.data_ptr()) if lse_h is not None else None, ctypes.byref(ticket))
        _capi.check(st, "host_step_run")
        t = int(ticket.value)
        self._keep[t] = (q_h, k_new_h, v_new_h, out_h, lse_h)
        for old in [k for k in self._keep if k < t - 1]:
            del self._keep[old]  # slot reused: that step has finished
        self.h2d_bytes = (cu.nbytes + sk.nbytes + bt.nbytes + T * 8
                          + 2 * T * (self.hq + 2 * self.hkv) * self.D)
        self.d2h_bytes = 2 * T * self.hq * self.D + (4 * T * self.hq if lse_h is not None else 0)
        return t

    def wait(self, ticket: int):
        from . import _capi

        _capi.check(self._lib.mcp_host_step_wait(self._h, int(ticket)), "host_step_wait")
        self._keep.pop(int(ticket), None)

    def __call__(self, q_h, k_new_h, v_new_h, cu_seqlens_q, seqlens_k, block_tables, k_cache,
                 v_cache, out_h, lse_h=None):
        self.wait(self.run(q_h, k_new_h, v_new_h, cu_seqlens_q, seqlens_k, block_tables,
                           k_cache, v_cache, out_h, lse_h))
        return out_h

    def close(self):
        from . import _capi

        if getattr(self, "_h", None) is not None and self._h.value:
            h, self._h = self._h, None
            _capi.check(self._lib.mcp_host_step_destroy(h), "host_step_destroy")
            self._keep.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
