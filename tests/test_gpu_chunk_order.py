"""Chunk operators on the GPU: what must not depend on which warp, stream or call comes first.  Batches, the plain form
and the tolerances are those of test_gpu_chunk.py."""
import pytest
import torch

from test_gpu_chunk import BF, F32, Batch, _ctx, _i32

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


def _keep_busy(products=60):
    """Work on the current stream, about 0.7 ms a product."""
    a = torch.ones(8192, 8192, device="cuda", dtype=BF)
    for _ in range(products):
        a = torch.matmul(a, a).mul_(2.0 ** -13)
    return a


@pytest.mark.parametrize("native", [True, False])
def test_outputs_a_call_allocates_for_a_side_stream_are_ordered_with_it(native):
    """No `out`, a stream of its own and a current stream that is far behind: nothing of the call, the zero fill of its
    outputs included, may be queued on the current stream."""
    b = Batch([(1, 90), (40, 200), (3, 3)], 8, 2, 128, BF, 16, seed=4, pad=3)
    k, v = (torch.randn(b.T, 2, 128, device="cuda").to(BF) for _ in range(2))
    prefix, new, free, head = _i32([0, 5, 9]), _i32([7, 0, 20]), torch.arange(8, dtype=torch.int32, device="cuda"), _i32([0])
    with _ctx(8, 2, 128, BF, n=3, pages=b.max_pages) as ctx:
        if not native:
            ctx._marshal = None

        def calls(**kw):
            table = b.table.clone() if not kw else tables
            p = ctx.plan(prefix, new, table, free, head, page_size=16, n_pages=b.pool.shape[0], max_rows=33, **kw)
            pool = b.pool.clone() if not kw else pools
            q = ctx.qk_norm_rope(b.q, k, v, pool, 0, p_rows, p_slots, **kw)
            return [p.row_offsets, p.kv_len, p.row_req, p.row_pos, p.row_slot, p.free_next, q, b.run(ctx, **kw)]

        p_rows, p_slots = torch.arange(b.T, dtype=torch.int32, device="cuda"), torch.full((b.T,), -1, dtype=torch.int32, device="cuda")
        tables, pools = b.table.clone(), b.pool.clone()
        want = calls()
        busy = _keep_busy()                                     # (loads the products' kernels)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            busy = _keep_busy()
            late = torch.cuda.Event()
            late.record()
            got = calls(stream=side)
            side.synchronize()
            assert not late.query()                             # the current stream is behind: the calls did not wait for it
            with torch.cuda.stream(side):
                seen = [t.cpu() for t in got]
            torch.cuda.synchronize()
            after = [t.cpu() for t in got]
            for w, s, a in zip(want, seen, after):
                assert torch.equal(s, w.cpu()) and torch.equal(a, w.cpu())
        assert ctx.device_error() == (0, 0) and bool(torch.isfinite(busy.float()).all())


@pytest.mark.parametrize("name", ["tiny", "small_bf16"])
@pytest.mark.parametrize("call", ["step", "decode_block"])
def test_outputs_a_step_allocates_for_a_side_stream_are_ordered_with_it(name, call):
    import focus_synth as fs
    from decodability_aware_token_b200 import FocusContext, StepParams
    from gpu_harness import limits_for, step_params, to_device
    case = fs.make_case(name)
    params = step_params(case.work)
    lim = limits_for(case, params)
    lim["max_keep"] = case.work.block                            # (decode_block's dense calls keep every position)
    with FocusContext(case.shape, to_device(case), **lim) as ctx:
        run, sp = getattr(ctx, call), StepParams(**params)
        batch = lambda: {k: v.cuda().clone() for k, v in case.batch.items()}
        outputs = lambda r: (r if call == "step" else r[0]).tensors()
        first = outputs(run(batch(), sp))
        torch.cuda.synchronize()
        want, flags = {k: t.cpu() for k, t in first.items()}, ctx.device_error()
        # (the case's page table ends with the prefix: a decoded block has no page to be committed to)
        assert flags[1] in ((0,) if call == "step" else (0, 0x2, 0x4))
        del first
        _keep_busy()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        b = batch()
        torch.cuda.synchronize()
        busy = _keep_busy(60 if call == "step" else 900)       # (a block is a few dozen steps, each read by the host)
        late = torch.cuda.Event()
        late.record()
        got = outputs(run(b, sp, stream=side))
        side.synchronize()
        assert not late.query()
        torch.cuda.synchronize()
        assert ctx.device_error() == flags and bool(torch.isfinite(busy.float()).all())
        for k, t in got.items():
            assert torch.equal(t.cpu(), want[k]), k


@pytest.mark.parametrize("S", [16, 64])
def test_an_engine_on_its_own_stream_prefills_what_the_current_stream_prepared(S):
    """The caller's tensors are written late on the current stream, dropped when the call returns, and their memory
    is written again at once."""
    import focus_synth as fs
    from decodability_aware_token_b200 import ChunkContext, FocusContext, StepParams
    from decodability_aware_token_b200.scheduler import FocusEngine
    from gpu_harness import to_device
    case = fs.make_case("small_bf16")
    s, lens = case.shape, [37, 64, 5, 100]
    N, mp = len(lens), 8
    g = torch.Generator().manual_seed(8)
    host = torch.randint(0, s.vocab, (N, max(lens)), generator=g, dtype=torch.int32)
    need = [-(-n // S) for n in lens]
    with FocusContext(s, to_device(case), max_requests=8, max_block=64, max_keep=64, max_pages_per_req=mp) as ctx, \
            ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                         max_requests=N, max_pages_per_req=mp, rope_theta=s.rope_theta) as chunk:
        def run(stream):
            eng = FocusEngine(ctx, StepParams(), stream=stream, chunk=chunk)
            pool = torch.zeros(sum(need) + 1, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=BF, device="cuda")
            view = dict(prefix_len=torch.full((N,), 3, dtype=torch.int32, device="cuda"), kv_pool=pool,
                        page_table=torch.full((N, mp), -1, dtype=torch.int32, device="cuda"))
            ids = [x.cuda() for x in (host, torch.tensor(lens, dtype=torch.int32), torch.arange(sum(need), dtype=torch.int32))]
            torch.cuda.synchronize()
            if stream is not None:
                _keep_busy()
            view["prefix_len"].zero_()
            args = [torch.empty_like(x).copy_(x) for x in ids]
            eng.prefill(view, *args)
            shapes = [a.shape for a in args]
            del args
            trash = [torch.full(sh, 7, dtype=torch.int32, device="cuda") for sh in shapes for _ in range(3)]
            got = (view["prefix_len"].tolist(), view["page_table"].cpu(), pool.cpu())   # (read on the current stream)
            assert ctx.device_error() == (0, 0) and chunk.device_error() == (0, 0) and len(trash) == 9
            return got
        want = run(None)
        assert want[0] == lens
        for _ in range(3):
            got = run(torch.cuda.Stream())
            assert got[0] == want[0] and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_the_scheduler_with_an_engine_on_its_own_stream():
    import focus_synth as fs
    from decodability_aware_token_b200 import ChunkContext, FocusContext, StepParams
    from decodability_aware_token_b200.scheduler import EffectiveBatchScheduler, FocusEngine, Request
    from gpu_harness import to_device
    case = fs.make_case("small_bf16", k_min=1, k_max=4)
    s, w, model = case.shape, case.work, to_device(case)
    B, S, mp, slots = 16, 16, 10, 4
    g = torch.Generator().manual_seed(19)
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (37, 1, 90, 20, 5)]

    def run(stream):
        pool = torch.zeros(60, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=BF, device="cuda")
        with FocusContext(s, model, max_requests=slots, max_block=B, max_keep=B, max_pages_per_req=mp) as ctx, \
                ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                             max_requests=slots, max_pages_per_req=mp, rope_theta=s.rope_theta) as chunk:
            eng = FocusEngine(ctx, StepParams(w.tau, w.k_min, w.k_max, w.conf_threshold, w.alpha), stream=stream, chunk=chunk,
                              mask_block=B)
            sch = EffectiveBatchScheduler(eng, slots=slots, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads,
                                          head_dim=s.head_dim, max_pages_per_req=mp, kv_pool=pool, free_pages=list(range(60)),
                                          mask_token=s.vocab - 1, k_max=w.k_max, keep_pages=True)
            for r, toks in enumerate(prompts):
                sch.submit(Request(r, r, len(toks), [], 2, prompt_tokens=toks))
            res = sch.run(max_iterations=500)
            assert ctx.device_error() == (0, 0) and chunk.device_error() == (0, 0)
            return {r: ([b.tolist() for b in x.blocks], x.steps, x.pages) for r, x in res.items()}, pool.cpu()
    want, pool = run(None)
    got, pool2 = run(torch.cuda.Stream())
    assert got == want and torch.equal(pool, pool2)
