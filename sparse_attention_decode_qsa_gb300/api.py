"""Python binding of the QSA decode-step library: same names as the C ABI
(include/qsa.h), argument marshalling only.  Every step of the decode path
runs in the CUDA library; PyTorch only allocates the device and pinned host
buffers and supplies the stream.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _native as N
from ._native import QsaError, check  # noqa: F401  (re-exported)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream_of(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the current stream of a device (by its index) as an address, without the
# Stream object around it (2 us of a call's 15 in Python)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _batch(handles, layer0: int, n_layers: int):
    arr = (N.Handle * len(handles))(*[N.Handle(h.index, h.generation) for h in handles])
    b = N.Batch(len(handles), layer0, n_layers, 0, C.cast(arr, C.POINTER(N.Handle)))
    b._keep = arr
    return b


def _chunk(handles, n_tokens, layer0: int, n_layers: int):
    n = len(handles)
    if len(n_tokens) != n:
        raise ValueError("one token count per request")
    # (assigned arrays are kept alive by the structure)
    return N.Chunk(n, layer0, n_layers, 0, (N.Handle * n)(*handles), (C.c_int32 * n)(*n_tokens))


class HostMemory:
    """Host memory from qsa_host_alloc: pages on a host NUMA node, mapped into
    the device's page tables and the host's at one address.  Pass
    .cpu(shape) as a request's host_rows; .cuda(shape) is a view of the same
    bytes for device-side copies.  Freed by free() (or when collected)."""

    def __init__(self, nbytes: int, device: int = 0, numa_node: int = -1):
        self.L = N.lib()
        out = C.c_void_p()
        check(self.L.qsa_host_alloc(int(device), int(numa_node), int(nbytes), C.byref(out)),
              "qsa_host_alloc")
        self.ptr, self.nbytes, self.device = out.value, int(nbytes), int(device)

    def cpu(self, shape) -> torch.Tensor:
        import numpy as np
        n = 1
        for x in shape:
            n *= int(x)
        if n > self.nbytes:
            raise ValueError("view larger than the allocation")
        arr = np.ctypeslib.as_array((C.c_uint8 * n).from_address(self.ptr)).reshape(tuple(shape))
        t = torch.from_numpy(arr)
        t._qsa_host_memory = self          # the view keeps the allocation alive
        return t

    def cuda(self, shape) -> torch.Tensor:
        n = 1
        for x in shape:
            n *= int(x)
        if n > self.nbytes:
            raise ValueError("view larger than the allocation")

        class _View:
            __cuda_array_interface__ = {"shape": tuple(int(x) for x in shape), "typestr": "|u1",
                                        "data": (self.ptr, False), "version": 3, "strides": None}
        t = torch.as_tensor(_View(), device=torch.device("cuda", self.device))
        t._qsa_host_memory = self
        return t

    def free(self):
        if getattr(self, "ptr", None):
            check(self.L.qsa_host_free(self.ptr), "qsa_host_free")
            self.ptr = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Cache:
    """A qsa_cache plus the device storage it runs on.

    With device=None the cache is host-only (bookkeeping without a GPU).
    Storage layout (all owned here, passed to the library as raw pointers):
      pool         uint8 [hbm_pool_rows][row_bytes] (2048 BF16 rows, 1040 FP8 rows)
      index_keys   uint8 [max_requests][n_layers][ctx_capacity][64]
      index_scales fp16  [max_requests][n_layers][ctx_capacity]
      slot_table   int32 [max_requests][n_layers][ctx_capacity]
      workspace    uint8 [qsa_workspace_bytes]
    hot_rows > 0 gives every offloaded request that many hot rows per layer
    (the cross-step hot cache filled by hot_cache_fetch).
    """

    def __init__(self, n_layers: int, max_requests: int, ctx_capacity: int,
                 hbm_pool_rows: int, budget_tokens: int = 2048, ring_tokens: int = 4096,
                 staging_rows: int = 2048, device="cuda", kv_format: int = N.KV_BF16,
                 hot_rows: int = 0):
        self.L = N.lib()
        cfg = N.CacheConfig()
        cfg.n_layers = n_layers
        cfg.max_requests = max_requests
        cfg.ctx_capacity = ctx_capacity
        cfg.budget_tokens = budget_tokens
        cfg.ring_tokens = ring_tokens
        cfg.staging_rows = staging_rows
        cfg.hbm_pool_rows = hbm_pool_rows
        cfg.kv_format = kv_format
        cfg.hot_rows = hot_rows
        self.kv_format = kv_format
        self.hot_rows = hot_rows
        self.row_bytes = N.ROW_BYTES_FP8 if kv_format == N.KV_FP8 else N.ROW_BYTES
        self.n_layers, self.max_requests, self.ctx_capacity = n_layers, max_requests, ctx_capacity
        self.budget_tokens, self.ring_tokens, self.staging_rows = budget_tokens, ring_tokens, staging_rows
        self.device = device
        if device is not None:
            ws = self.L.qsa_workspace_bytes(C.byref(cfg))
            if ws < 0:
                raise QsaError(N.ERR_INVALID_ARG, "qsa_workspace_bytes", "bad config")
            self.pool = torch.empty(hbm_pool_rows, self.row_bytes, dtype=torch.uint8, device=device)
            self.index_keys = torch.zeros(max_requests, n_layers, ctx_capacity, N.INDEX_DIM,
                                          dtype=torch.uint8, device=device)
            self.index_scales = torch.zeros(max_requests, n_layers, ctx_capacity,
                                            dtype=torch.float16, device=device)
            self.slot_table = torch.empty(max_requests, n_layers, ctx_capacity,
                                          dtype=torch.int32, device=device)
            self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)
            cfg.hbm_pool = self.pool.data_ptr()
            cfg.index_keys = self.index_keys.data_ptr()
            cfg.index_scales = self.index_scales.data_ptr()
            cfg.slot_table = self.slot_table.data_ptr()
            cfg.workspace = self.workspace.data_ptr()
            cfg.workspace_bytes = ws
        self.cfg = cfg
        h = C.c_void_p()
        check(self.L.qsa_cache_create(C.byref(cfg), C.byref(h)), "qsa_cache_create")
        self.h = h
        self._host = {}

    def close(self):
        if getattr(self, "h", None):
            self.L.qsa_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------- bookkeeping
    def request_begin(self, ctx_len: int, placement: int = N.KV_HBM, host_rows=None,
                      stream=None, max_ctx: int = 0) -> N.Handle:
        """Lease a request of ctx_len tokens that may grow to max_ctx (0: no
        growth).  host_rows: pinned host history [n_layers][max(ctx_len,
        max_ctx)][2048] for the host placements."""
        d = N.RequestDesc(ctx_len, placement, max_ctx, None)
        if host_rows is not None:
            d.host_rows = host_rows.data_ptr() if isinstance(host_rows, torch.Tensor) else int(host_rows)
        out = N.Handle()
        check(self.L.qsa_request_begin(self.h, C.byref(d), self._current(stream), C.byref(out)), "qsa_request_begin")
        if isinstance(host_rows, torch.Tensor):
            self._host[out.index] = host_rows
        return out

    def request_end(self, handle: N.Handle):
        check(self.L.qsa_request_end(self.h, handle), "qsa_request_end")
        self._host.pop(handle.index, None)

    def request_info(self, handle: N.Handle) -> N.RequestInfo:
        out = N.RequestInfo()
        check(self.L.qsa_request_info_get(self.h, handle, C.byref(out)), "qsa_request_info_get")
        return out

    def advance(self, handle: N.Handle, n_new: int = 1):
        """Reserve the positions of n_new new tokens (ctx_len grows by n_new)."""
        check(self.L.qsa_request_advance(self.h, handle, n_new), "qsa_request_advance")

    def stats(self) -> dict:
        out = N.Stats()
        check(self.L.qsa_cache_stats(self.h, C.byref(out)), "qsa_cache_stats")
        return out.as_dict()

    def slot_table_ptr(self, handle: N.Handle, layer: int) -> int:
        out = C.c_void_p()
        check(self.L.qsa_slot_table_ptr(self.h, handle, layer, C.byref(out)), "qsa_slot_table_ptr")
        return out.value

    def slot_table_set(self, handle: N.Handle, layer: int, tokens, slots, stream=None):
        check(self.L.qsa_slot_table_set(self.h, handle, layer, _ptr(tokens), _ptr(slots),
                                        int(tokens.numel()), _stream(stream)), "qsa_slot_table_set")

    def staging_ptr(self, layer: int) -> int:
        out = C.c_void_p()
        check(self.L.qsa_staging_ptr(self.h, layer, C.byref(out)), "qsa_staging_ptr")
        return out.value

    def poll_error(self, stream=None):
        st, det = C.c_int32(), C.c_int64()
        check(self.L.qsa_poll_error(self.h, _stream(stream), C.byref(st), C.byref(det)),
              "qsa_poll_error")
        return st.value, det.value

    # -------------------------------------------------- pages of the cache
    def truncate(self, handle: N.Handle, ctx_len: int):
        """Take back the newest tokens: the request's context becomes ctx_len."""
        check(self.L.qsa_request_truncate(self.h, handle, int(ctx_len)), "qsa_request_truncate")

    def request_fork(self, parent: N.Handle, ctx_len: int, placement: int = N.KV_HBM, host_rows=None,
                     stream=None, max_ctx: int = 0) -> N.Handle:
        """Lease a request that starts with the first ctx_len tokens of
        `parent` (copied: keys, rows), with the placement, host history and
        growth that request_begin takes."""
        d = N.RequestDesc(ctx_len, placement, max_ctx, None)
        if host_rows is not None:
            d.host_rows = host_rows.data_ptr() if isinstance(host_rows, torch.Tensor) else int(host_rows)
        out = N.Handle()
        check(self.L.qsa_request_fork(self.h, parent, C.byref(d), self._current(stream), C.byref(out)),
              "qsa_request_fork")
        if isinstance(host_rows, torch.Tensor):
            self._host[out.index] = host_rows
        return out

    def compact(self, stream=None) -> int:
        """Close the gaps of the pool; returns the number of rows moved."""
        moved = C.c_int64()
        check(self.L.qsa_cache_compact(self.h, self._current(stream), C.byref(moved)), "qsa_cache_compact")
        return moved.value

    # ------------------------------------------------------ producer side
    def append_token(self, handles, layer0, n_layers, k_new, kv_new, stream=None):
        """Store each unit's newest token: k_new fp32 [units][64] index keys,
        kv_new uint8 [units][2048] KV rows (unit u = i_layer * n_req + i_req)."""
        b = _batch(handles, layer0, n_layers)
        check(self.L.qsa_append_token(self.h, C.byref(b), _ptr(k_new), _ptr(kv_new),
                                      _stream(stream)), "qsa_append_token")

    # ---------------------------------------------------------- hot path
    def index_score(self, handles, layer0, n_layers, q_idx, w, blk_scores, stream=None):
        b = _batch(handles, layer0, n_layers)
        check(self.L.qsa_index_score(self.h, C.byref(b), _ptr(q_idx), _ptr(w), _ptr(blk_scores),
                                     blk_scores.shape[-1], _stream(stream)), "qsa_index_score")

    def select_c4_topk(self, handles, layer0, n_layers, blk_scores, budget_tokens, sel_blocks,
                       n_sel, stream=None):
        b = _batch(handles, layer0, n_layers)
        check(self.L.qsa_select_c4_topk(self.h, C.byref(b), _ptr(blk_scores), blk_scores.shape[-1],
                                        budget_tokens, _ptr(sel_blocks), _ptr(n_sel),
                                        _stream(stream)), "qsa_select_c4_topk")

    def gather_rows(self, handles, layer0, n_layers, sel_blocks, n_sel, budget_tokens, rows_out,
                    n_rows=None, stream=None):
        b = _batch(handles, layer0, n_layers)
        out_ptr = rows_out if isinstance(rows_out, int) else _ptr(rows_out)
        check(self.L.qsa_gather_rows(self.h, C.byref(b), _ptr(sel_blocks), _ptr(n_sel),
                                     budget_tokens, out_ptr, _ptr(n_rows), _stream(stream)),
              "qsa_gather_rows")

    def hot_cache_fetch(self, handles, layer0, n_layers, sel_blocks, n_sel, budget_tokens,
                        stream=None):
        b = _batch(handles, layer0, n_layers)
        check(self.L.qsa_hot_cache_fetch(self.h, C.byref(b), _ptr(sel_blocks), _ptr(n_sel),
                                         budget_tokens, _stream(stream)), "qsa_hot_cache_fetch")

    def hot_cache_plan(self, handles, layer0, n_layers, sel_blocks, n_sel, budget_tokens,
                       stream=None):
        b = _batch(handles, layer0, n_layers)
        check(self.L.qsa_hot_cache_plan(self.h, C.byref(b), _ptr(sel_blocks), _ptr(n_sel),
                                        budget_tokens, _stream(stream)), "qsa_hot_cache_plan")

    def sparse_decode_attn(self, handles, layer0, n_layers, q, sel_blocks, n_sel, budget_tokens,
                           gathered, softmax_scale, out, lse=None, stream=None):
        b = _batch(handles, layer0, n_layers)
        g = gathered if (gathered is None or isinstance(gathered, int)) else _ptr(gathered)
        check(self.L.qsa_sparse_decode_attn(self.h, C.byref(b), _ptr(q.view(torch.int16)),
                                            _ptr(sel_blocks), _ptr(n_sel), budget_tokens, g,
                                            float(softmax_scale), _ptr(out), _ptr(lse),
                                            _stream(stream)), "qsa_sparse_decode_attn")

    def _rows(self, t, what, dtypes, shape):
        """Address of a per-row tensor (None: a null pointer).  Its type, shape,
        device and layout are checked here, since the library sees an address."""
        if t is None:
            return None
        if t.dtype not in dtypes:
            raise ValueError(f"{what}: type {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if t.shape != shape:
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {shape}")
        if self.device is not None and t.device != self.pool.device:
            raise ValueError(f"{what}: on {t.device}, the cache on {self.pool.device}")
        return _ptr(t)

    def _current(self, stream):
        """The stream given, else the current one of the cache's device (a cache
        without device storage takes none)."""
        if self.device is None:
            return None
        return _raw_stream(self.pool.device.index) if stream is None else _stream(stream)

    # ------------------------------------------------ several tokens at once
    # handles: requests; n_tokens: how many of each request's newest tokens.
    # Rows: layer after layer, request after request.
    def append_chunk(self, handles, n_tokens, layer0, n_layers, k_new, kv_new, stream=None):
        """Store the chunk's tokens: k_new fp32 [rows][64], kv_new uint8 [rows][2048]."""
        ch = _chunk(handles, n_tokens, layer0, n_layers)
        rows = n_layers * sum(n_tokens)
        check(self.L.qsa_append_chunk(self.h, C.byref(ch),
                                      self._rows(k_new, "k_new", (torch.float32,), (rows, N.INDEX_DIM)),
                                      self._rows(kv_new, "kv_new", (torch.uint8,), (rows, N.ROW_BYTES)),
                                      self._current(stream)), "qsa_append_chunk")

    def chunk_index_score(self, handles, n_tokens, layer0, n_layers, q_idx, w, blk_scores, stream=None):
        """Block scores of every query: q_idx fp32 or bf16 [rows][8][64], w fp32
        [rows][8], blk_scores fp32 [rows][stride]."""
        ch = _chunk(handles, n_tokens, layer0, n_layers)
        rows = n_layers * sum(n_tokens)
        check(self.L.qsa_chunk_index_score(
            self.h, C.byref(ch),
            self._rows(q_idx, "q_idx", (torch.float32, torch.bfloat16), (rows, N.INDEX_HEADS, N.INDEX_DIM)),
            N.QUERY_BF16 if q_idx.dtype == torch.bfloat16 else N.QUERY_F32,
            self._rows(w, "w", (torch.float32,), (rows, N.INDEX_HEADS)),
            self._rows(blk_scores, "blk_scores", (torch.float32,), (rows, blk_scores.shape[-1])), blk_scores.shape[-1],
            self._current(stream)), "qsa_chunk_index_score")

    def chunk_select_topk(self, handles, n_tokens, layer0, n_layers, blk_scores, budget_tokens,
                          sel_blocks, n_sel, stream=None):
        """Best blocks of every query: sel_blocks int32 [rows][budget/4], n_sel int32 [rows]."""
        ch = _chunk(handles, n_tokens, layer0, n_layers)
        rows = n_layers * sum(n_tokens)
        check(self.L.qsa_chunk_select_topk(
            self.h, C.byref(ch), self._rows(blk_scores, "blk_scores", (torch.float32,), (rows, blk_scores.shape[-1])),
            blk_scores.shape[-1], budget_tokens,
            self._rows(sel_blocks, "sel_blocks", (torch.int32,), (rows, budget_tokens // 4)),
            self._rows(n_sel, "n_sel", (torch.int32,), (rows,)), self._current(stream)), "qsa_chunk_select_topk")

    def chunk_attn_workspace_bytes(self, handles, n_tokens, layer0, n_layers, budget_tokens) -> int:
        ch = _chunk(handles, n_tokens, layer0, n_layers)
        n = self.L.qsa_chunk_attn_workspace_bytes(self.h, C.byref(ch), budget_tokens)
        if n < 0:
            raise QsaError(N.ERR_INVALID_ARG, "qsa_chunk_attn_workspace_bytes",
                           self.L.qsa_last_error_string().decode(errors="replace"))
        return n

    def chunk_sparse_attn(self, handles, n_tokens, layer0, n_layers, q, sel_blocks, n_sel, budget_tokens,
                          softmax_scale, out, lse=None, workspace=None, stream=None):
        """Attention of every query over its own blocks: q and out bf16
        [rows][16][128], lse fp32 [rows][16].  workspace: uint8 of
        chunk_attn_workspace_bytes bytes; allocated for the call when None."""
        ch = _chunk(handles, n_tokens, layer0, n_layers)
        rows = n_layers * sum(n_tokens)
        if workspace is None:
            need = self.chunk_attn_workspace_bytes(handles, n_tokens, layer0, n_layers, budget_tokens)
            # allocated in the order of the stream that uses it: memory of the
            # current stream may still be at work there
            if stream is not None and not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=self.pool.device)
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=self.pool.device)
        heads = (rows, N.Q_HEADS, N.HEAD_DIM)
        check(self.L.qsa_chunk_sparse_attn(
            self.h, C.byref(ch), self._rows(q, "q", (torch.bfloat16,), heads),
            self._rows(sel_blocks, "sel_blocks", (torch.int32,), (rows, budget_tokens // 4)),
            self._rows(n_sel, "n_sel", (torch.int32,), (rows,)), budget_tokens, float(softmax_scale),
            self._rows(out, "out", (torch.bfloat16,), heads),
            self._rows(lse, "lse", (torch.float32,), (rows, N.Q_HEADS)),
            self._rows(workspace, "workspace", (torch.uint8,), (workspace.numel(),)), workspace.numel(),
            self._current(stream)), "qsa_chunk_sparse_attn")
