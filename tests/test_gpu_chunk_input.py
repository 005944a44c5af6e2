"""Chunk operators on the GPU: input that is at the edge of what the header allows, or beyond it.  Batches, the plain form
and the tolerances are those of test_gpu_chunk.py."""
import pytest
import torch

from test_gpu_chunk import BF, F32, Batch, _ctx, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("n", [40, 2])
def test_row_offsets_that_go_back_skip_their_request_and_no_other(dt, d, n):
    """Ranges around a decreasing pair overlap (rows of two requests are undefined); those of one request come out right."""
    S, part = 16, n // 2
    b = Batch([(n, 90 + r) for r in range(3)], 8, 2, d, dt, S, seed=n, pad=part * 2)
    offs = [0, n, part, part + n, 2 * part, 2 * part + n]       # 0 .. n, back, part .. part + n, back, 2 part .. 2 part + n
    lens = [90, 5, 91, 5, 92]
    table = b.table[[0, 0, 1, 1, 2]].contiguous()
    with _ctx(8, 2, d, dt, n=5, pages=b.max_pages) as ctx:
        want = []
        for r in range(3):                                      # each request alone, its rows where they are in the batch
            one = Batch.__new__(Batch)
            one.__dict__.update(b.__dict__)
            one.reqs, one.offs, one.table = [(n, 90 + r)], [r * part, r * part + n], b.table[r:r + 1]
            one.row_offsets, one.kv_len = _i32(one.offs), _i32([90 + r])
            out = one.run(ctx)
            one.check(out)
            want.append(out)
        assert ctx.device_error() == (0, 0)
        out = torch.full_like(b.q, 5.0)
        ctx.attention(b.q, b.pool, 1, _i32(offs), _i32(lens), table, out=out)
        torch.cuda.synchronize()
        assert ctx.device_error() == (-5, 0x20)
        first, last = slice(0, part), slice(n + part, n + 2 * part)
        tol = 2.0 ** -7 if dt == BF else 1e-5                   # (another split of the walk: sums in another order)
        for rows, w in ((first, want[0]), (last, want[2])):
            assert float((out[rows].float() - w[rows].float()).abs().max()) <= tol * float(w[rows].float().abs().max())
        assert bool((out[n + 2 * part:] == 5).all())


@pytest.mark.parametrize("lag,top", [(30, 60), (33, 63), (-30, 63)])
@pytest.mark.parametrize("reqs,hq,hkv", [
    ([(200, 700), (1, 600), (300, 300), (150, 64 + 150)], 8, 2),   # whole walks and pieces
    ([(40, 9000)], 4, 1), ([(3, 9000)], 4, 1),                      # one unit over many CTAs, tile and few-row kernel
])
def test_attention_of_large_values_under_a_reference_that_lags(reqs, hq, hkv, lag, top):
    """The first 64 keys score about 0, the others about `lag` in units of log2: 64 weights of 2^lag sum to less than
    the 2^40 that raises the tile kernel's reference, and are summed with values of magnitude 2^top as they are."""
    S, d = 32, 128
    b = Batch(reqs, hq, hkv, d, BF, S, seed=lag + top, gain=0.05)
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.sign(torch.randn(d, generator=g, device="cuda"))
    b.q += u.to(BF)
    table = b.table.cpu()
    for r, (_, kv) in enumerate(reqs):
        for i in range(-(-kv // S)):
            m = min(S, kv - i * S)
            along = (0.0 if i * S < 64 else lag) * 0.6931471805599453 / d ** 0.5
            page = b.pool[int(table[r, i])]
            page[:, 0, :, :m] = (along * u + 0.02 * torch.randn(m, d, generator=g, device="cuda")).to(BF)
            page[:, 1, :, :m] = (page[:, 1, :, :m].float().clamp(-1, 1) * 2.0 ** top).to(BF)
    with _ctx(hq, hkv, d, BF, n=len(reqs), pages=b.max_pages) as ctx:
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0) and bool(torch.isfinite(out.float()).all())
        b.check(out)
