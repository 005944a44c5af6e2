"""Chunk operators on the GPU where a batch is unusual: thousands of requests most of which have nothing to do, scores
that climb from block to block, graphs that share a context, a captured prefill.  Batches, the plain form and the
tolerances are those of test_gpu_chunk.py."""
import pytest
import torch

from test_gpu_chunk import BF, F32, Batch, _ctx, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("N,live", [
    (300, {0: (1, 40), 150: (70, 200), 299: (1, 9)}),                       # more requests than threads of a block
    (3000, {7: (1, 300), 8: (33, 33), 1500: (300, 301), 1501: (1, 1), 2999: (5, 70)}),
    (16384, {0: (90, 95), 9000: (1, 500), 16383: (2, 2)}),                  # the limit
    (1000, {b: (1 + b % 3, 1 + b % 150) for b in range(0, 1000, 2)}),       # every other request
])
def test_attention_of_many_requests_most_of_them_idle(dt, d, N, live):
    reqs = [live.get(b, (0, 0)) for b in range(N)]
    reqs = [(n, max(n, kv)) for n, kv in reqs]
    b = Batch(reqs, 8, 2, d, dt, 16, seed=N, pad=2)
    with _ctx(8, 2, d, dt, n=N, pages=b.max_pages) as ctx:
        out = torch.full_like(b.q, 5.0)
        b.run(ctx, out=out)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        b.check(out)
        assert bool((out[b.offs[-1]:] == 5).all())


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("climb", [1.5, -1.5, 0.2])
def test_attention_scores_that_climb_from_block_to_block(dt, d, climb):
    """Scores that change by `climb` a key (in units of log2: 96 a block of 64) leave the range of any reference taken
    from an earlier block; falling ones leave later blocks without weight."""
    reqs = [(1, 450), (1, 40), (150, 420), (300, 300), (4, 600)]
    b = Batch(reqs, 8, 2, d, dt, 16, seed=5, gain=0.1)
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.sign(torch.randn(d, generator=g, device="cuda"))             # |u|^2 = d
    b.q += u.to(dt)                                                        # q . u = d + noise
    table = b.table.cpu()
    for r, (_, kv) in enumerate(reqs):
        for i in range(-(-kv // 16)):
            page = int(table[r, i])
            pos = torch.arange(i * 16, min(kv, i * 16 + 16), device="cuda", dtype=torch.float32)
            # scale q . K = climb pos / log2(e), scale = 1 / sqrt(d)
            along = climb * pos * 0.6931471805599453 / d ** 0.5
            b.pool[page, :, 0, :, : len(pos)] = (along[:, None] * u + 0.05 * torch.randn(len(pos), d, generator=g, device="cuda")).to(dt)
    with _ctx(8, 2, d, dt, n=len(reqs), pages=b.max_pages) as ctx:
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        b.check(out)


def test_attention_large_values_stay_in_range():
    """Values up to 2^60 with weights that grow to the edge of what one reference covers."""
    b = Batch([(1, 500), (200, 200)], 4, 2, 128, BF, 32, seed=9)
    b.pool[:, :, 1] *= 2.0 ** 58
    with _ctx(4, 2, 128, BF, n=2, pages=b.max_pages) as ctx:
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0) and bool(torch.isfinite(out.float()).all())
        b.check(out)


@pytest.mark.parametrize("hq,hkv", [(7, 1), (21, 3), (50, 1)])
def test_attention_groups_that_do_not_divide_the_tile_after_one_with_nan(hq, hkv):
    """Tile rows that no query vector fills hold whatever an earlier kernel left: here rows of NaN."""
    reqs = [(60, 200), (33, 90)]
    nan, b = Batch(reqs, 8, 1, 128, BF, 64, seed=1), Batch(reqs, hq, hkv, 128, BF, 64, seed=2)
    nan.q.fill_(float("nan"))
    with _ctx(8, 1, 128, BF, n=2, pages=nan.max_pages) as first, _ctx(hq, hkv, 128, BF, n=2, pages=b.max_pages) as ctx:
        bad = nan.run(first)
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert bool(torch.isnan(bad).all())
        assert ctx.device_error() == (0, 0)
        b.check(out)


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
def test_two_graphs_of_one_context_replayed_in_turn(dt, d):
    one = Batch([(1, 900), (1, 30), (50, 700)], 8, 2, d, dt, 16, seed=1, slack=3)
    two = Batch([(200, 260), (1, 1), (1, 800)], 8, 2, d, dt, 16, seed=2, slack=3)
    pages = max(one.max_pages, two.max_pages)
    for b in (one, two):
        b.table = torch.nn.functional.pad(b.table, (0, pages - b.max_pages), value=-1)
    with _ctx(8, 2, d, dt, n=3, pages=pages) as ctx:
        want = [b.run(ctx).clone() for b in (one, two)]
        outs, graphs = [torch.zeros_like(w) for w in want], []
        for b, o in zip((one, two), outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                b.run(ctx, out=o)
            graphs.append(g)
        for i in range(40):
            graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        one.check(outs[0]), two.check(outs[1])


@pytest.mark.parametrize("name", ["tiny", "small_bf16"])
def test_captured_prefill_does_what_the_eager_one_does(name):
    from test_gpu_prefill import Model
    lens = [40, 9, 0, 33]
    eager, m = Model(name, lens, 16), Model(name, lens, 16)
    plan = eager.run(lens, max_rows=90)
    eager.ok()
    tok = torch.zeros(4, max(lens), dtype=torch.int32)
    for b, t in enumerate(m.tokens):
        tok[b, : len(t)] = torch.tensor(t, dtype=torch.int32)
    tok, new, out = tok.cuda(), _i32(lens), m.chunk.alloc_plan(4, 90)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.ctx.prefill(m.chunk, tok, new, m.batch, m.free, m.head, out=out)
    for _ in range(3):  # each replay starts from empty prefixes
        m.batch["prefix_len"].zero_()
        m.batch["page_table"].fill_(-1)
        m.pool.fill_(float("nan"))
        g.replay()
    m.ok()
    assert m.batch["prefix_len"].tolist() == lens and out.row_offsets.tolist() == plan.row_offsets.tolist()
    assert torch.equal(m.batch["page_table"], eager.batch["page_table"])
    # the same bits, NaN in the same untouched places
    assert torch.equal(m.pool.nan_to_num(nan=123.0), eager.pool.nan_to_num(nan=123.0))
    # a second chunk of one request by another replay, the others idle
    new.copy_(_i32([0, 5, 0, 0]))
    m.free.copy_(torch.roll(m.free, -int(out.free_next)))
    g.replay()
    m.ok()
    assert m.batch["prefix_len"].tolist() == [40, 14, 0, 33]
    del g
    m.close(), eager.close()


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("bad", [0, 1, 2, 3])
def test_a_nan_query_row_is_nan_and_no_other_is(dt, d, bad):
    """Walks that are split over CTAs and walks that are not: the row comes out as NaN, its neighbours as they are."""
    reqs = [(1, 5000), (1, 3), (70, 2000), (20, 20)]
    b = Batch(reqs, 8, 2, d, dt, 16, seed=3)
    row = b.offs[bad] + (reqs[bad][0] - 1) // 2
    with _ctx(8, 2, d, dt, n=4, pages=b.max_pages) as ctx:
        want = b.run(ctx)
        b.q[row] = float("nan")
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        assert bool(torch.isnan(out[row]).all())
        keep = torch.arange(b.T, device="cuda") != row
        assert torch.equal(out[keep], want[keep])
