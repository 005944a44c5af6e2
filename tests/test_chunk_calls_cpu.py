"""Chunk operators, host side: arguments at the edge of their types, and a context that is closed more than once (no GPU)."""
import ctypes as C

import pytest
import torch

from decodability_aware_token_b200 import ChunkContext, FocusContext, FocusError, _abi
from test_chunk_cpu import HKV, HQ, D, L, MAXP, PAGES, S, _ctx


def test_a_scale_that_float32_cannot_hold_is_refused():
    """The C struct's float32 scale has 0 stand for 1 / sqrt(d): a scale that rounds to it is not the default."""
    calls = []
    ctx = _ctx(calls=calls)
    i32 = dict(dtype=torch.int32)
    a = dict(q=torch.zeros(4, HQ, D), kv_pool=torch.zeros(PAGES, L, 2, HKV, S, D), layer=2,
             row_offsets=torch.zeros(3, **i32), kv_len=torch.zeros(2, **i32), page_table=torch.zeros(2, MAXP, **i32))
    for scale in (1e-50, 1e-320, 1e39, float("inf"), float("nan"), -1.0, 0.0, -1e-50):
        with pytest.raises(ValueError):
            ctx.attention(**a, scale=scale)
    assert not calls
    for scale in (1.5e-45, 1e-38, 0.25, 3e38):
        ctx.attention(**a, scale=scale)
        assert _abi.ChunkAttnArgs.from_buffer_copy(calls[-1][1]).scale == C.c_float(scale).value > 0


@pytest.mark.parametrize("cls,fn", [(ChunkContext, "focus_chunk_destroy"), (FocusContext, "focus_destroy")])
@pytest.mark.parametrize("rc", [_abi.FOCUS_OK, _abi.FOCUS_ERR_CUDA])
def test_a_context_is_destroyed_once_whatever_the_status(cls, fn, rc):
    """The library frees the context also when it reports an error: nothing may be handed to it again."""
    seen = []

    class Lib:
        pass
    setattr(Lib, fn, lambda self, ctx: (seen.append(ctx.value), rc)[1])
    ctx = cls.__new__(cls)
    ctx._ctx, ctx._lib = C.c_void_p(0x1000), Lib()
    if rc:
        with pytest.raises(FocusError):
            ctx.close()
    ctx.close()
    ctx.close()
    del ctx
    assert seen == [0x1000]
