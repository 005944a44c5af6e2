"""Prompt chunks over the paged KV cache: pages and rows for new tokens, query/key norm with rotation and
cache write, attention over everything a request has cached.

The focused step reads prefix pages that already hold a prompt's keys and values; these operators fill them.
Like the rest of the package this module only marshals arguments for the C ABI (include/focus.h); the
computation is in the library's kernels.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import math
from typing import Optional

import torch

from . import _abi, _check, _need, _under

__all__ = ["ChunkContext", "ChunkPlan"]


_I32 = torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


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
    only the outputs they are not given, and can be captured in CUDA graphs.  Outputs are allocated on that stream: a
    consumer on another one waits for it, as for any tensor made under torch.cuda.stream.  Two calls of one
    context must not overlap in time; use a context per concurrent stream.
    """
    _marshal = None

    def __init__(self, *, n_layers: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                 max_requests: int, max_pages_per_req: int, rope_theta: float = 10000.0, device="cuda"):
        self._ctx = C.c_void_p()
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"dtype {dtype}: expected torch.bfloat16 or torch.float32")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"device {dev}: a CUDA device is needed")
        self._lib = _abi.load()
        self._enqueue = _abi.load_enqueue()
        self._marshal, self._entry = _abi.load_marshal()
        self.device = torch.device("cuda", torch.cuda.current_device() if dev.index is None else dev.index)
        self.dtype = dtype
        self._index = self.device.index
        self._elt = 2 if dtype == torch.bfloat16 else 4
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
    # A call whose outputs are given and whose device is current goes through csrc/marshal.cpp, which makes the
    # checks below in C++ and returns None where one fails.  The Python path then makes them again: the fast tests
    # decide, _need and _heads_error word the refusal.
    def _stream(self, stream, where):
        if not self._ctx.value:
            raise ValueError(f"{where}: the context is closed")
        if stream is None:
            return _raw_stream(self._index)
        if stream.device_index != self._index:
            raise ValueError(f"{where}: the stream is on cuda:{stream.device_index}, the context on {self.device}")
        return stream.cuda_stream

    def _ints(self, t, name, shape):
        if not (isinstance(t, torch.Tensor) and t.dtype is _I32 and t.get_device() == self._index and
                t.shape == shape and t.is_contiguous()):
            _need(t, name, _I32, self.device, shape)
        return t.data_ptr()

    def _heads(self, t, name, rows, heads):
        """[rows, heads, d] with dense heads; returns (data pointer, row stride in elements)."""
        d = self.head_dim
        if not (isinstance(t, torch.Tensor) and t.dtype is self.dtype and t.get_device() == self._index and
                t.shape == (rows, heads, d)):
            self._heads_error(t, name, rows, heads)
        s0, s1, s2 = t.stride()
        if rows <= 1:
            s0 = heads * d  # the stride of a single row means nothing
        p = t.data_ptr()
        if s2 != 1 or (s1 != d and heads > 1):
            raise ValueError(f"{name}: the heads of a row must be dense")
        if s0 < heads * d:
            raise ValueError(f"{name}: rows overlap (stride {s0})")
        if p % 16 or s0 * self._elt % 16:
            raise ValueError(f"{name}: rows must be 16-byte aligned")
        return p, s0

    def _heads_error(self, t, name, rows, heads):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        if t.dtype != self.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {self.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, expected {self.device}")
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({rows}, {heads}, {self.head_dim})")

    def _pool(self, pool, layer):
        if not (isinstance(pool, torch.Tensor) and pool.dtype is self.dtype and pool.get_device() == self._index and
                pool.is_contiguous()):
            _need(pool, "kv_pool", self.dtype, self.device)
        s, L = pool.shape, self.cfg.n_layers
        if len(s) != 6 or s[1:4] != (L, 2, self.n_kv_heads) or s[5] != self.head_dim:
            raise ValueError(f"kv_pool: shape {tuple(s)}, expected [pages, {L}, 2, {self.n_kv_heads}, S, {self.head_dim}]")
        if not 0 <= layer < L:
            raise ValueError(f"layer {layer}: the pool has {L}")
        p = pool.data_ptr()
        if p % 16:
            raise ValueError("kv_pool: must be 16-byte aligned")
        return s[0], s[4], p

    def _call(self, which, args, where, stream):
        fn, s = self._enqueue[which], self._stream(stream, where)
        if _current_device() == self._index:
            rc = fn(self._ctx, args, s)
        else:
            with torch.cuda.device(self.device):
                rc = fn(self._ctx, args, s)
        if rc:
            _check(rc, where)

    # ---- operators --------------------------------------------------------------------------------------
    def plan(self, prefix_len, new_len, page_table, free_pages, free_head, *, page_size: int, n_pages: int,
             max_rows: Optional[int] = None, out: Optional[ChunkPlan] = None,
             stream: Optional[torch.cuda.Stream] = None) -> ChunkPlan:
        """Give every request of a chunk its pages and rows, first come, first served (focus_chunk_plan_rows).

        prefix_len, new_len [N] int32; page_table [N, max_pages_per_req] int32, new pages are written into it;
        free_pages [F] int32, taken from index free_head [1] int32 on.  `max_rows` (or the size of `out`)
        bounds the rows.  A request that does not fit gets no rows: row_offsets tells."""
        where = "focus_chunk_plan_rows"
        if self._marshal and out is not None and max_rows is None and _current_device() == self._index:
            rc = self._marshal.plan(
                self._entry[0], self._ctx.value, self._stream(stream, where), self._index, self.limits.max_pages_per_req,
                page_size, n_pages, prefix_len, new_len, page_table, free_pages, free_head, out.row_offsets, out.kv_len,
                out.row_req, out.row_pos, out.row_slot, out.free_next)
            if rc == 0:
                return out
            if rc is not None:
                _check(rc, where)
        args, out = self._plan_args(prefix_len, new_len, page_table, free_pages, free_head, page_size, n_pages, max_rows, out,
                                    stream)
        self._call(0, args, where, stream)
        return out

    def _plan_args(self, prefix_len, new_len, page_table, free_pages, free_head, page_size, n_pages, max_rows, out,
                   stream=None):
        n = prefix_len.shape[0]
        if out is None:
            if max_rows is None:
                raise ValueError("plan: give max_rows or out")
            with _under(stream):
                out = self.alloc_plan(n, max_rows)
        rows = out.row_req.shape[0]
        if max_rows is not None and max_rows != rows:
            raise ValueError(f"plan: out holds {rows} rows, max_rows is {max_rows}")
        i, per_req, per_row, n_free = self._ints, (n,), (rows,), free_pages.shape[0]
        return _abi.PLAN_PACK.pack(
            n, rows, page_size, n_pages, n_free, i(prefix_len, "prefix_len", per_req), i(new_len, "new_len", per_req),
            i(page_table, "page_table", (n, self.limits.max_pages_per_req)), i(free_pages, "free_pages", (n_free,)),
            i(free_head, "free_head", (1,)), i(out.row_offsets, "row_offsets", (n + 1,)), i(out.kv_len, "kv_len", per_req),
            i(out.row_req, "row_req", per_row), i(out.row_pos, "row_pos", per_row), i(out.row_slot, "row_slot", per_row),
            i(out.free_next, "free_next", (1,))), out

    def qk_norm_rope(self, q, k, v, kv_pool, layer: int, row_pos, row_slot, *, q_norm=None, k_norm=None,
                     eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Norm (with the gains given), rotate, store K and V at row_slot; returns the queries
        (focus_chunk_qk_norm_rope).  q [rows, Hq, d], k and v [rows, Hkv, d] may be views of one fused
        projection; rows with row_pos < 0 are skipped."""
        where = "focus_chunk_qk_norm_rope"
        if self._marshal and out is not None and _current_device() == self._index:
            rc = self._marshal.qk(
                self._entry[1], self._ctx.value, self._stream(stream, where), self._index, self._elt == 2, self.n_q_heads,
                self.n_kv_heads, self.head_dim, self.cfg.n_layers, layer, eps, q, k, v, kv_pool, row_pos, row_slot, q_norm,
                k_norm, out)
            if rc == 0:
                return out
            if rc is not None:
                _check(rc, where)
        rows, hq, hkv = q.shape[0], self.n_q_heads, self.n_kv_heads
        qp, qs = self._heads(q, "q", rows, hq)
        kp, ks = self._heads(k, "k", rows, hkv)
        vp, vs = self._heads(v, "v", rows, hkv)
        if out is None:
            with _under(stream):
                out = torch.zeros(rows, hq, self.head_dim, dtype=self.dtype, device=self.device)
        op, os_ = self._heads(out, "out", rows, hq)
        n_pages, page_size, pool = self._pool(kv_pool, layer)
        gq = self._gain(q_norm, "q_norm") if q_norm is not None else 0
        gk = self._gain(k_norm, "k_norm") if k_norm is not None else 0
        args = _abi.QK_PACK.pack(rows, layer, page_size, n_pages, eps, qs, ks, vs, os_, qp, kp, vp, gq, gk,
                                 self._ints(row_pos, "row_pos", (rows,)), self._ints(row_slot, "row_slot", (rows,)), op, pool)
        self._call(1, args, where, stream)
        return out

    def _gain(self, t, name):
        if not (isinstance(t, torch.Tensor) and t.dtype is self.dtype and t.get_device() == self._index and
                t.shape == (self.head_dim,) and t.is_contiguous()):
            _need(t, name, self.dtype, self.device, (self.head_dim,))
        p = t.data_ptr()
        if p % 16:
            raise ValueError(f"{name}: must be 16-byte aligned")
        return p

    def attention(self, q, kv_pool, layer: int, row_offsets, kv_len, page_table, *, max_new: Optional[int] = None,
                  mask_block: int = 1, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the chunk's queries [rows, Hq, d] over the cached keys and values
        (focus_chunk_attention).  `max_new` bounds the rows of a request (default: all rows); a tight bound
        saves work.  mask_block 1 is the causal mask, B the block-causal mask of blocks of B positions."""
        where = "focus_chunk_attention"
        if scale is not None and not 0 < C.c_float(scale).value < math.inf:  # (0 would stand for 1 / sqrt(d))
            raise ValueError(f"scale {scale}: must be positive and finite in float32")
        if self._marshal and out is not None and max_new is not None and _current_device() == self._index:
            rc = self._marshal.attention(
                self._entry[2], self._ctx.value, self._stream(stream, where), self._index, self._elt == 2, self.n_q_heads,
                self.n_kv_heads, self.head_dim, self.cfg.n_layers, self.limits.max_pages_per_req, layer, max_new, mask_block,
                0.0 if scale is None else scale, q, kv_pool, row_offsets, kv_len, page_table, out)
            if rc == 0:
                return out
            if rc is not None:
                _check(rc, where)
        rows, n, hq = q.shape[0], kv_len.shape[0], self.n_q_heads
        qp, qs = self._heads(q, "q", rows, hq)
        if out is None:
            with _under(stream):
                out = torch.zeros(rows, hq, self.head_dim, dtype=self.dtype, device=self.device)
        op, os_ = self._heads(out, "out", rows, hq)
        n_pages, page_size, pool = self._pool(kv_pool, layer)
        if max_new is None:
            max_new = max(rows, 1)
        i, row = self._ints, (n, self.limits.max_pages_per_req)
        args = _abi.ATTN_PACK.pack(n, rows, max_new, page_size, n_pages, layer, mask_block, 0.0 if scale is None else scale,
                                   qs, os_, qp, pool, i(row_offsets, "row_offsets", (n + 1,)), i(kv_len, "kv_len", (n,)),
                                   i(page_table, "page_table", row), op)
        self._call(2, args, where, stream)
        return out

    # ---- state ------------------------------------------------------------------------------------------
    def device_error(self):
        """Synchronise, read and clear the device error word -> (status code, FOCUS_DEVERR_* bits)."""
        bits = C.c_int32(0)
        rc = self._lib.focus_chunk_get_device_error(self._ctx, C.byref(bits))
        return rc, bits.value

    def close(self):
        if getattr(self, "_ctx", None) is not None and self._ctx.value:
            ctx, self._ctx = self._ctx, C.c_void_p()  # (freed whatever the status is)
            _check(self._lib.focus_chunk_destroy(ctx), "focus_chunk_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
