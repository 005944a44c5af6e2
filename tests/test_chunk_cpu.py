"""Chunk operators, host side: packed argument layout, refusals of the binding and of the C ABI (no GPU).

The binding's checks run on CPU tensors against a context that was never initialised on a device: its calls
are recorded instead of made."""
import ctypes as C

import pytest
import torch

from decodability_aware_token_b200 import ChunkContext, ChunkPlan, _abi

HQ, HKV, D, L, S, PAGES, MAXP = 4, 2, 64, 3, 5, 7, 6


def _ctx(dtype=torch.float32, calls=None):
    ctx = ChunkContext.__new__(ChunkContext)
    ctx._ctx = C.c_void_p()
    ctx.device, ctx._index, ctx.dtype = torch.device("cpu"), -1, dtype
    ctx._elt = 2 if dtype == torch.bfloat16 else 4
    ctx.cfg = _abi.ChunkCfg(L, HQ, HKV, D, _abi.FOCUS_DTYPE_F32, 1e4)
    ctx.limits = _abi.ChunkLimits(8, MAXP)
    ctx.n_q_heads, ctx.n_kv_heads, ctx.head_dim = HQ, HKV, D
    ctx._call = lambda which, args, where, stream: (calls if calls is not None else []).append((which, args))
    return ctx


@pytest.mark.parametrize("pack,mirror", [(_abi.PLAN_PACK, _abi.ChunkPlanArgs), (_abi.QK_PACK, _abi.ChunkQkArgs),
                                         (_abi.ATTN_PACK, _abi.ChunkAttnArgs)])
def test_packed_arguments_have_the_struct_layout(pack, mirror):
    fields = mirror._fields_
    assert pack.size == C.sizeof(mirror)
    vals = [float(i + 1) if t is C.c_float else i + 1 for i, (_, t) in enumerate(fields)]
    got = mirror.from_buffer_copy(pack.pack(*vals))
    assert [getattr(got, n) for n, _ in fields] == vals


def _plan_args(n=3, rows=9):
    i32 = dict(dtype=torch.int32)
    return dict(prefix_len=torch.zeros(n, **i32), new_len=torch.ones(n, **i32), page_table=torch.zeros(n, MAXP, **i32),
                free_pages=torch.arange(4, **i32), free_head=torch.zeros(1, **i32))


def test_plan_marshals_and_refuses():
    calls = []
    ctx = _ctx(calls=calls)
    a = _plan_args()
    out = ctx.plan(**a, page_size=S, n_pages=PAGES, max_rows=9)
    got = _abi.ChunkPlanArgs.from_buffer_copy(calls[0][1])
    assert (got.n_requests, got.max_rows, got.page_size, got.n_pages, got.n_free) == (3, 9, S, PAGES, 4)
    assert got.page_table == a["page_table"].data_ptr() and got.row_slot == out.row_slot.data_ptr()
    assert out.row_offsets.shape == (4,) and out.kv_len.shape == (3,) and out.row_req.shape == (9,)
    with pytest.raises(ValueError):
        ctx.plan(**a, page_size=S, n_pages=PAGES)                                   # neither rows nor out
    with pytest.raises(ValueError):
        ctx.plan(**a, page_size=S, n_pages=PAGES, max_rows=8, out=out)              # out of another size
    for key, bad, exc in (("new_len", torch.ones(2, dtype=torch.int32), ValueError),
                          ("new_len", torch.ones(3, dtype=torch.int64), TypeError),
                          ("page_table", torch.zeros(3, MAXP + 1, dtype=torch.int32), ValueError),
                          ("page_table", torch.zeros(MAXP, 3, dtype=torch.int32).t(), ValueError),
                          ("free_head", torch.zeros(2, dtype=torch.int32), ValueError)):
        with pytest.raises(exc):
            ctx.plan(**{**a, key: bad}, page_size=S, n_pages=PAGES, max_rows=9)
    short = ChunkPlan(out.row_offsets[:3], out.kv_len, out.row_req, out.row_pos, out.row_slot, out.free_next)
    with pytest.raises(ValueError):
        ctx.plan(**a, page_size=S, n_pages=PAGES, out=short)


def _qk_args(rows=4):
    qkv = torch.zeros(rows, HQ + 2 * HKV, D)
    return dict(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:], kv_pool=torch.zeros(PAGES, L, 2, HKV, S, D),
                layer=1, row_pos=torch.zeros(rows, dtype=torch.int32), row_slot=torch.zeros(rows, dtype=torch.int32))


def test_qk_marshals_strided_views_and_refuses():
    calls = []
    ctx = _ctx(calls=calls)
    a = _qk_args()
    out = ctx.qk_norm_rope(**a, eps=0.5)
    got = _abi.ChunkQkArgs.from_buffer_copy(calls[0][1])
    assert (got.rows, got.layer, got.page_size, got.n_pages, got.eps) == (4, 1, S, PAGES, 0.5)
    assert got.q_stride == got.k_stride == got.v_stride == (HQ + 2 * HKV) * D and got.out_stride == HQ * D
    assert got.k == a["q"].data_ptr() + HQ * D * 4 and not got.q_norm and out.shape == (4, HQ, D)
    big = torch.zeros(4, HQ, 2 * D)
    flat = torch.zeros(4 * HQ * D + 1)
    for key, bad, exc in (("k", a["q"], ValueError),                               # wrong head count
                          ("q", a["q"].to(torch.bfloat16), TypeError),
                          ("q", big[:, :, ::2], ValueError),                       # elements not dense
                          ("q", big[:, :, :D], ValueError),                        # heads not dense
                          ("q", flat[1:].view(4, HQ, D), ValueError),              # not 16-byte aligned
                          ("q", torch.zeros(1, HQ, D).expand(4, HQ, D), ValueError),  # rows overlap
                          ("v", a["v"][:3], ValueError),
                          ("kv_pool", torch.zeros(PAGES, L, 2, HKV, S, D + 1), ValueError),
                          ("kv_pool", torch.zeros(PAGES, L + 1, 2, HKV, S, D), ValueError),
                          ("layer", L, ValueError), ("layer", -1, ValueError),
                          ("row_slot", torch.zeros(3, dtype=torch.int32), ValueError),
                          ("row_pos", torch.zeros(4), TypeError)):
        with pytest.raises(exc):
            ctx.qk_norm_rope(**{**a, key: bad})
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(**a, q_norm=torch.ones(D + 1))
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(**a, out=torch.zeros(5, HQ, D))


def test_attention_marshals_and_refuses():
    calls = []
    ctx = _ctx(calls=calls)
    i32 = dict(dtype=torch.int32)
    a = dict(q=torch.zeros(4, HQ, D), kv_pool=torch.zeros(PAGES, L, 2, HKV, S, D), layer=2,
             row_offsets=torch.zeros(3, **i32), kv_len=torch.zeros(2, **i32), page_table=torch.zeros(2, MAXP, **i32))
    ctx.attention(**a, mask_block=16, max_new=3)
    got = _abi.ChunkAttnArgs.from_buffer_copy(calls[0][1])
    assert (got.n_requests, got.rows, got.max_new, got.page_size, got.n_pages, got.layer, got.mask_block) == \
        (2, 4, 3, S, PAGES, 2, 16) and got.scale == 0.0
    ctx.attention(**a)
    assert _abi.ChunkAttnArgs.from_buffer_copy(calls[1][1]).max_new == 4
    for key, bad, exc in (("row_offsets", torch.zeros(2, **i32), ValueError), ("kv_len", torch.zeros(2), TypeError),
                          ("page_table", torch.zeros(2, MAXP - 1, **i32), ValueError), ("layer", 3, ValueError)):
        with pytest.raises(exc):
            ctx.attention(**{**a, key: bad})
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError):
            ctx.attention(**a, scale=scale)
    with pytest.raises(ValueError):
        ctx.attention(**a, out=torch.zeros(3, HQ, D))


def test_context_refuses_before_the_device():
    kw = dict(n_layers=1, n_q_heads=4, n_kv_heads=2, head_dim=128, max_requests=1, max_pages_per_req=1)
    with pytest.raises(TypeError):
        ChunkContext(**kw, dtype=torch.float16, device="cuda:0")
    with pytest.raises(ValueError):
        ChunkContext(**kw, device="cpu")


def _cfg(**over):
    base = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=_abi.FOCUS_DTYPE_BF16, rope_theta=1e4)
    base.update(over)
    return _abi.ChunkCfg(**base)


@pytest.mark.parametrize("over,lim,code", [
    (dict(n_layers=0), (4, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(n_q_heads=7), (4, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(dtype=5), (4, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(rope_theta=0.0), (4, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(rope_theta=float("inf")), (4, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(), (0, 4), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(), (4, 0), _abi.FOCUS_ERR_INVALID_ARG),
    (dict(head_dim=64), (4, 4), _abi.FOCUS_ERR_UNSUPPORTED),
    (dict(head_dim=96, dtype=_abi.FOCUS_DTYPE_F32), (4, 4), _abi.FOCUS_ERR_UNSUPPORTED),
    (dict(n_q_heads=130, n_kv_heads=2), (4, 4), _abi.FOCUS_ERR_UNSUPPORTED),
    (dict(), (16385, 4), _abi.FOCUS_ERR_LIMITS),
])
def test_chunk_init_refuses_before_the_device(over, lim, code):
    lib = _abi.load()
    ctx = C.c_void_p(1)
    assert lib.focus_chunk_init(C.byref(_cfg(**over)), C.byref(_abi.ChunkLimits(*lim)), C.byref(ctx)) == code
    assert not ctx.value
    if code != _abi.FOCUS_ERR_LIMITS:
        assert lib.focus_chunk_workspace_bytes(C.byref(_cfg(**over)), C.byref(_abi.ChunkLimits(*lim))) == 0


def test_chunk_null_handles_are_safe():
    lib = _abi.load()
    assert lib.focus_chunk_init(None, None, None) == _abi.FOCUS_ERR_INVALID_ARG
    assert lib.focus_chunk_destroy(None) == _abi.FOCUS_OK
    assert lib.focus_chunk_get_device_error(None, None) == _abi.FOCUS_ERR_INVALID_ARG
    assert lib.focus_chunk_plan_rows(None, None, None) == _abi.FOCUS_ERR_INVALID_ARG
    assert lib.focus_chunk_qk_norm_rope(None, None, None) == _abi.FOCUS_ERR_INVALID_ARG
    assert lib.focus_chunk_attention(None, None, None) == _abi.FOCUS_ERR_INVALID_ARG
    assert lib.focus_chunk_workspace_bytes(C.byref(_cfg()), C.byref(_abi.ChunkLimits(4, 4))) > 0
