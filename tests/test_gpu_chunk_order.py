"""Chunk operators on the GPU: what must not depend on which warp, stream or call comes first.  Batches, the plain form
and the tolerances are those of test_gpu_chunk.py."""
import pytest
import torch

from test_gpu_chunk import F32, Batch, _ctx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,S", [(64, 16), (64, 24), (128, 16), (128, 7)])
def test_float32_walks_of_many_blocks_repeat_themselves(d, S):
    """Chunks over many key blocks with pages that are not mapped and a partial last block: each block's keys are told
    from the missing ones by its own marks, however far apart the warps of a CTA run."""
    reqs = [(70, 70 + 17 * 64 + 5), (33, 900), (64, 64), (128, 1301), (1, 777), (200, 3 * 64 + 1)]
    b = Batch(reqs, 8, 2, d, F32, S, seed=d + S)
    missing = {}
    for r, i in ((0, 3), (0, 40), (1, 0), (3, 17), (3, 18), (5, 2)):
        if i >= -(-reqs[r][1] // S):
            continue
        b.table[r, i] = -1
        missing.setdefault(r, set()).update(range(i * S, min(i * S + S, reqs[r][1])))
    with _ctx(8, 2, d, F32, n=len(reqs), pages=b.max_pages) as ctx:
        first = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (-5, 0x2)
        b.check(first, missing=missing)
        outs = [b.run(ctx) for _ in range(60)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
