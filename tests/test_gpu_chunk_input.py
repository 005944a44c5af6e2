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


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("native", [True, False])
def test_outputs_that_overlap_the_inputs_are_refused(dt, native):
    from decodability_aware_token_b200 import FocusError
    hq, hkv, d, T = 4, 2, 128, 6
    b = Batch([(T, 20)], hq, hkv, d, dt, 16, seed=1)
    pos, slot = torch.arange(T, dtype=torch.int32, device="cuda"), torch.full((T,), -1, dtype=torch.int32, device="cuda")
    wide = torch.randn(T + 2, 3 * hq + 2 * hkv, d, device="cuda").to(dt)          # q | k | v | two outputs' worth
    q, k, v, rest = wide[:T, :hq], wide[:T, hq:hq + hkv], wide[:T, hq + hkv:hq + 2 * hkv], hq + 2 * hkv
    flat = lambda t, at, n: t.flatten()[at:at + n * hq * d].view(n, hq, d)
    whole = lambda n: wide.as_strided((n, hq, d), (hq * d, d, 1))                   # dense rows over the same memory
    bad_qk = {"a head on": wide[:T, 1:hq + 1], "a row on": wide[1:T + 1, :hq], "into k": wide[:T, hq:2 * hq],
              "into v": wide[:T, hq + 1:2 * hq + 1], "a row on, into v": wide[1:T + 1, hq + hkv:2 * hq + hkv],
              "other stride": whole(T), "the pool": flat(b.pool, 0, T), "the pool's end": b.pool.flatten()[-T * hq * d:].view(T, hq, d)}
    good_qk = {"in place": q, "beside": wide[:T, rest:rest + hq], "beside, two rows on": wide[2:, rest + hq:], "apart": torch.zeros(T, hq, d, dtype=dt, device="cuda")}
    with _ctx(hq, hkv, d, dt, n=1, pages=b.max_pages) as ctx:
        if not native:
            ctx._marshal = None
        keep = wide.clone(), b.pool.nan_to_num(nan=3.0).clone()
        for what, out in bad_qk.items():
            with pytest.raises(FocusError) as e:
                ctx.qk_norm_rope(q, k, v, b.pool, 0, pos, slot, out=out)
            assert e.value.code == -1, what
            if what in ("into k", "into v", "a row on, into v"):
                continue
            with pytest.raises(FocusError) as e:
                ctx.attention(q, b.pool, 1, b.row_offsets, b.kv_len, b.table, max_new=T, out=out)
            assert e.value.code == -1, what
        with pytest.raises(FocusError):                                               # attention is not done in place
            ctx.attention(q, b.pool, 1, b.row_offsets, b.kv_len, b.table, max_new=T, out=q)
        torch.cuda.synchronize()
        assert torch.equal(wide, keep[0]) and torch.equal(b.pool.nan_to_num(nan=3.0), keep[1])
        want = ctx.qk_norm_rope(q, k, v, b.pool, 0, pos, slot)
        o = ctx.attention(q, b.pool, 1, b.row_offsets, b.kv_len, b.table)
        for what, out in good_qk.items():
            wide.copy_(keep[0])
            if what != "in place":
                assert torch.equal(ctx.attention(q, b.pool, 1, b.row_offsets, b.kv_len, b.table, max_new=T, out=out), o), what
            assert torch.equal(ctx.qk_norm_rope(q, k, v, b.pool, 0, pos, slot, out=out), want), what
            assert torch.equal(k, keep[0][:T, hq:hq + hkv]) and torch.equal(v, keep[0][:T, hq + hkv:hq + 2 * hkv])
        # a single row has no stride
        one = wide[:1, :hq]
        with pytest.raises(FocusError):
            ctx.qk_norm_rope(one, k[:1], v[:1], b.pool, 0, pos[:1], slot[:1], out=wide[:1, 2:hq + 2])
        ctx.qk_norm_rope(one, k[:1], v[:1], b.pool, 0, pos[:1], slot[:1], out=wide[:1, rest:rest + hq])
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
