"""Prompt chunks over the paged KV cache: pages and rows for new tokens, query/key norm with rotation and
cache write, attention over everything a request has cached.

The focused step reads prefix pages that already hold a prompt's keys and values; these operators fill them.
Like the rest of the package this module only marshals arguments for the C ABI (include/focus.h); the
computation is in the library's kernels.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
from typing import Optional

import torch

from . import _abi, _check, _need

__all__ = ["ChunkContext", "ChunkPlan"]


@dataclasses.dataclass
class ChunkPlan:
    """Where a chunk's tokens go: request b owns rows row_offsets[b] .. row_offsets[b + 1] - 1."""
    row_offsets: torch.Tensor      # [N + 1] int32
    kv_len: torch.Tensor           # [N] int32: cached tokens, the new ones included
    row_req: torch.Tensor          # [rows] int32, -1 past the last row
    row_pos: torch.Tensor          # [rows] int32, -1 past the last row
    row_slot: torch.Tensor         # [rows] int32: page * S + offset, -1 where there is none
    free_next: torch.Tensor        # [1] int32: free-list head after this plan


class ChunkContext:
    """The chunk operators of one model geometry: scratch, rotary frequencies and a device error word.

    Calls are asynchronous on `stream` (default: torch's current stream on the context's device), allocate
    only the outputs they are not given, and can be captured in CUDA graphs.  Two calls of one context must
    not overlap in time; use a context per concurrent stream.
    """

    def __init__(self, *, n_layers: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                 max_requests: int, max_pages_per_req: int, rope_theta: float = 10000.0, device="cuda"):
        self._ctx = C.c_void_p()
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"dtype {dtype}: expected torch.bfloat16 or torch.float32")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"device {dev}: a CUDA device is needed")
        self._lib = _abi.load()
        self.device = torch.device("cuda", torch.cuda.current_device() if dev.index is None else dev.index)
        self.dtype = dtype
        self.cfg = _abi.ChunkCfg(n_layers, n_q_heads, n_kv_heads, head_dim,
                                 _abi.FOCUS_DTYPE_BF16 if dtype == torch.bfloat16 else _abi.FOCUS_DTYPE_F32, rope_theta)
        self.limits = _abi.ChunkLimits(max_requests, max_pages_per_req)
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        with torch.cuda.device(self.device):
            _check(self._lib.focus_chunk_init(C.byref(self.cfg), C.byref(self.limits), C.byref(self._ctx)),
                   "focus_chunk_init")

    def workspace_bytes(self) -> int:
        return int(self._lib.focus_chunk_workspace_bytes(C.byref(self.cfg), C.byref(self.limits)))

    def alloc_plan(self, n: int, max_rows: int) -> ChunkPlan:
        kw = dict(dtype=torch.int32, device=self.device)
        return ChunkPlan(torch.zeros(n + 1, **kw), torch.zeros(n, **kw), torch.zeros(max_rows, **kw),
                         torch.zeros(max_rows, **kw), torch.zeros(max_rows, **kw), torch.zeros(1, **kw))

    # ---- checks -----------------------------------------------------------------------------------------
    def _ints(self, t, name, shape):
        _need(t, name, torch.int32, self.device, shape)
        return t.data_ptr()

    def _heads(self, t, name, heads):
        """[rows, heads, d] with dense heads; returns (data pointer, row stride in elements)."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        if t.dtype != self.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {self.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, expected {self.device}")
        d = self.head_dim
        if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [rows, {heads}, {d}]")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (s1 != d and heads > 1):
            raise ValueError(f"{name}: the heads of a row must be dense")
        if t.shape[0] <= 1:
            s0 = heads * d  # the stride of a single row means nothing
        if s0 < heads * d:
            raise ValueError(f"{name}: rows overlap (stride {s0})")
        if t.data_ptr() % 16 or s0 * t.element_size() % 16:
            raise ValueError(f"{name}: rows must be 16-byte aligned")
        return t.data_ptr(), s0

    def _pool(self, pool, layer):
        _need(pool, "kv_pool", self.dtype, self.device)
        s = pool.shape
        if pool.dim() != 6 or s[1] != self.cfg.n_layers or s[2] != 2 or s[3] != self.n_kv_heads or s[5] != self.head_dim:
            raise ValueError(f"kv_pool: shape {tuple(s)}, expected [pages, {self.cfg.n_layers}, 2, {self.n_kv_heads}, S, "
                             f"{self.head_dim}]")
        if not 0 <= layer < self.cfg.n_layers:
            raise ValueError(f"layer {layer}: the pool has {self.cfg.n_layers}")
        return s[0], s[4], pool.data_ptr()

    def _call(self, fn, args, where, stream):
        if self._ctx.value is None:
            raise ValueError(f"{where}: the context is closed")
        if torch.cuda.current_device() == self.device.index:
            s = stream.cuda_stream if stream is not None else torch.cuda.current_stream().cuda_stream
            _check(fn(self._ctx, C.byref(args), s), where)
        else:
            with torch.cuda.device(self.device):
                s = stream.cuda_stream if stream is not None else torch.cuda.current_stream().cuda_stream
                _check(fn(self._ctx, C.byref(args), s), where)

    # ---- operators --------------------------------------------------------------------------------------
    def plan(self, prefix_len, new_len, page_table, free_pages, free_head, *, page_size: int, n_pages: int,
             max_rows: Optional[int] = None, out: Optional[ChunkPlan] = None,
             stream: Optional[torch.cuda.Stream] = None) -> ChunkPlan:
        """Give every request of a chunk its pages and rows, first come, first served (focus_chunk_plan_rows).

        prefix_len, new_len [N] int32; page_table [N, max_pages_per_req] int32, new pages are written into it;
        free_pages [F] int32, taken from index free_head [1] int32 on.  `max_rows` (or the size of `out`)
        bounds the rows.  A request that does not fit gets no rows: row_offsets tells."""
        n = int(prefix_len.shape[0])
        if out is None:
            if max_rows is None:
                raise ValueError("plan: give max_rows or out")
            out = self.alloc_plan(n, max_rows)
        rows = int(out.row_req.shape[0])
        if max_rows is not None and max_rows != rows:
            raise ValueError(f"plan: out holds {rows} rows, max_rows is {max_rows}")
        i = self._ints
        args = _abi.ChunkPlanArgs(
            n, rows, page_size, n_pages, int(free_pages.shape[0]), i(prefix_len, "prefix_len", (n,)),
            i(new_len, "new_len", (n,)), i(page_table, "page_table", (n, self.limits.max_pages_per_req)),
            i(free_pages, "free_pages", (int(free_pages.shape[0]),)), i(free_head, "free_head", (1,)),
            i(out.row_offsets, "row_offsets", (n + 1,)), i(out.kv_len, "kv_len", (n,)), i(out.row_req, "row_req", (rows,)),
            i(out.row_pos, "row_pos", (rows,)), i(out.row_slot, "row_slot", (rows,)),
            i(out.free_next, "free_next", (1,)))
        self._call(self._lib.focus_chunk_plan_rows, args, "focus_chunk_plan_rows", stream)
        return out

    def qk_norm_rope(self, q, k, v, kv_pool, layer: int, row_pos, row_slot, *, q_norm=None, k_norm=None,
                     eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Norm (with the gains given), rotate, store K and V at row_slot; returns the queries
        (focus_chunk_qk_norm_rope).  q [rows, Hq, d], k and v [rows, Hkv, d] may be views of one fused
        projection; rows with row_pos < 0 are skipped."""
        rows = int(q.shape[0])
        qp, qs = self._heads(q, "q", self.n_q_heads)
        kp, ks = self._heads(k, "k", self.n_kv_heads)
        vp, vs = self._heads(v, "v", self.n_kv_heads)
        if k.shape[0] != rows or v.shape[0] != rows:
            raise ValueError(f"k, v: {k.shape[0]}, {v.shape[0]} rows, q has {rows}")
        if out is None:
            out = torch.zeros(rows, self.n_q_heads, self.head_dim, dtype=self.dtype, device=self.device)
        elif out.shape[0] != rows:
            raise ValueError(f"out: {out.shape[0]} rows, q has {rows}")
        op, os_ = self._heads(out, "out", self.n_q_heads)
        n_pages, page_size, pool = self._pool(kv_pool, layer)
        gains = []
        for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None:
                _need(t, name, self.dtype, self.device, (self.head_dim,))
                if t.data_ptr() % 16:
                    raise ValueError(f"{name}: must be 16-byte aligned")
            gains.append(t.data_ptr() if t is not None else None)
        args = _abi.ChunkQkArgs(rows, layer, page_size, n_pages, eps, qs, ks, vs, os_, qp, kp, vp, gains[0], gains[1],
                                self._ints(row_pos, "row_pos", (rows,)), self._ints(row_slot, "row_slot", (rows,)), op, pool)
        self._call(self._lib.focus_chunk_qk_norm_rope, args, "focus_chunk_qk_norm_rope", stream)
        return out

    def attention(self, q, kv_pool, layer: int, row_offsets, kv_len, page_table, *, max_new: Optional[int] = None,
                  mask_block: int = 1, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the chunk's queries [rows, Hq, d] over the cached keys and values
        (focus_chunk_attention).  `max_new` bounds the rows of a request (default: all rows); a tight bound
        saves work.  mask_block 1 is the causal mask, B the block-causal mask of blocks of B positions."""
        rows, n = int(q.shape[0]), int(kv_len.shape[0])
        qp, qs = self._heads(q, "q", self.n_q_heads)
        if out is None:
            out = torch.zeros(rows, self.n_q_heads, self.head_dim, dtype=self.dtype, device=self.device)
        elif out.shape[0] != rows:
            raise ValueError(f"out: {out.shape[0]} rows, q has {rows}")
        op, os_ = self._heads(out, "out", self.n_q_heads)
        n_pages, page_size, pool = self._pool(kv_pool, layer)
        if max_new is None:
            max_new = max(rows, 1)
        if scale is None:
            scale = 0.0
        elif not scale > 0:
            raise ValueError(f"scale {scale}: must be positive")
        args = _abi.ChunkAttnArgs(n, rows, max_new, page_size, n_pages, layer, mask_block, scale, qs, os_, qp, pool,
                                  self._ints(row_offsets, "row_offsets", (n + 1,)), self._ints(kv_len, "kv_len", (n,)),
                                  self._ints(page_table, "page_table", (n, self.limits.max_pages_per_req)), op)
        self._call(self._lib.focus_chunk_attention, args, "focus_chunk_attention", stream)
        return out

    # ---- state ------------------------------------------------------------------------------------------
    def device_error(self):
        """Synchronise, read and clear the device error word -> (status code, FOCUS_DEVERR_* bits)."""
        bits = C.c_int32(0)
        rc = self._lib.focus_chunk_get_device_error(self._ctx, C.byref(bits))
        return rc, bits.value

    def close(self):
        if getattr(self, "_ctx", None) is not None and self._ctx.value:
            _check(self._lib.focus_chunk_destroy(self._ctx), "focus_chunk_destroy")
            self._ctx = C.c_void_p()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
