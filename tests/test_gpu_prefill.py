"""Prompts through the whole model on the GPU (focus_prefill) against the float64 block-causal forward, and through
the scheduler, whose requests then decode what they decode with the same prompts already cached.

Tolerances are the step's own: max-abs error within 1e-4 x RMS (float32) and 2e-2 x RMS (bf16, four layers of
hidden 512) of the float64 values.  Cached values add the roundings they are stored with, at u = 2^-8 (2^-24 in
float32) relative: V one, u |v|; K two, the projection's row (x, y) before the turn and the result after it: a turn
passes on at most u (|x| + |y|) <= sqrt(2) u r and the store adds u r, r the pair's norm, which the turn keeps."""
import numpy as np
import pytest
import torch

import focus_synth as fs
from gpu_harness import to_device
from oracle import focus_oracle as fo
from prefill_reference import cached, prompt_forward

pytestmark = pytest.mark.gpu

FRAC = {"f32": 1e-4, "bf16": 2e-2}


def _close(got, want, dtype, what, stored=0.0):
    rms = float(np.sqrt(np.mean(want ** 2)))
    over = float((np.abs(got - want) - stored).max())
    assert over <= FRAC[dtype] * rms, f"{what}: {over:.3e} > {FRAC[dtype]} x RMS {rms:.3e}"


def _stored(want, dtype, turned):
    """What the stored roundings of K (turned) or V may add, elementwise."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    if not turned:
        return u * np.abs(want)
    lo, hi = np.split(want, 2, axis=-1)
    r = np.sqrt(lo * lo + hi * hi)
    return (1 + np.sqrt(2)) * u * np.concatenate([r, r], axis=-1)


class Model:
    def __init__(self, name, lens, S, slots=8, block=64, spare=6, seed=2):
        from decodability_aware_token_b200 import ChunkContext, FocusContext
        self.case = fs.make_case(name)
        s = self.shape = self.case.shape
        self.model = to_device(self.case)
        g = torch.Generator().manual_seed(seed)
        self.tokens = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in lens]
        self.lens, self.S, N = lens, S, len(lens)
        need = sum(-(-n // S) for n in lens)
        mp = max(-(-n // S) for n in lens) + 1
        dt = torch.bfloat16 if s.dtype == "bf16" else torch.float32
        self.pool = torch.full((need + spare, s.n_layers, 2, s.n_kv_heads, S, s.head_dim), float("nan"), dtype=dt, device="cuda")
        self.free = torch.randperm(need + spare, generator=g).to(torch.int32).cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.batch = dict(prefix_len=torch.zeros(N, dtype=torch.int32, device="cuda"), kv_pool=self.pool,
                          page_table=torch.full((N, mp), -1, dtype=torch.int32, device="cuda"))
        self.ctx = FocusContext(s, self.model, max_requests=slots, max_block=block, max_keep=block, max_pages_per_req=mp)
        self.chunk = ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                                  dtype=dt, max_requests=N, max_pages_per_req=mp, rope_theta=s.rope_theta)

    def run(self, new, **kw):
        """One chunk of `new[b]` tokens of each request, taken where its prefix ends."""
        done = self.batch["prefix_len"].tolist()
        tok = torch.zeros(len(new), max(max(new), 1), dtype=torch.int32)
        for b, n in enumerate(new):
            tok[b, :n] = torch.tensor(self.tokens[b][done[b]:done[b] + n], dtype=torch.int32)
        plan = self.ctx.prefill(self.chunk, tok.cuda(), torch.tensor(new, dtype=torch.int32).cuda(), self.batch, self.free,
                                self.head, **kw)
        self.head.copy_(plan.free_next)
        return plan

    def ok(self):
        torch.cuda.synchronize()
        assert self.ctx.device_error() == (0, 0) and self.chunk.device_error() == (0, 0)

    def close(self):
        self.ctx.close()
        self.chunk.close()


@pytest.mark.parametrize("name,S,lens,mask_block,splits", [
    ("tiny", 16, [20, 1, 33, 0, 16], 1, None), ("tiny", 5, [20, 7, 13], 4, [[8, 4, 12], [12, 3, 1]]),
    ("small_bf16", 16, [30, 1, 64, 17], 1, None), ("small_bf16", 64, [40, 33, 70], 32, [[32, 32, 64], [8, 1, 6]]),
    ("small_bf16", 32, [90, 64, 100, 81], 16, None),             # more than 256 rows: the many-row GEMMs
])
def test_prefill_matches_the_float64_forward(name, S, lens, mask_block, splits):
    m = Model(name, lens, S)
    D, rows = m.shape.hidden, sum(lens) + 3
    hidden = torch.zeros(rows, D, device="cuda")
    for new in splits or [lens]:
        plan = m.run(new, mask_block=mask_block, hidden=hidden, max_rows=rows)
        m.ok()
        offs = plan.row_offsets.tolist()
    assert m.batch["prefix_len"].tolist() == lens
    table = m.batch["page_table"].cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kv, hid = prompt_forward(m.shape, m.case.model, m.tokens[b], mask_block)
        got = cached(m.pool, table[b], n)
        for l in range(m.shape.n_layers):
            for i, what in enumerate(("K", "V")):
                _close(got[l, i], kv[l, i], m.shape.dtype, f"{what} of request {b}, layer {l}",
                       _stored(kv[l, i], m.shape.dtype, what == "K"))
        last = (splits or [lens])[-1][b]
        _close(hidden[offs[b]:offs[b] + last].cpu().double().numpy(), hid[n - last:], m.shape.dtype, f"hidden of {b}")
    # without `hidden` the last layer stops at its cache write, which is the same
    again = Model(name, lens, S)
    for new in splits or [lens]:
        again.run(new, mask_block=mask_block, max_rows=rows)
    again.ok()
    for b, n in enumerate(lens):
        np.testing.assert_array_equal(cached(again.pool, table[b], n), cached(m.pool, table[b], n))
    m.close(), again.close()


def test_prefill_with_head_norms():
    """Per-head gains: the keys of layer 0 are those of the operator's own formula on the layer's projection."""
    m = Model("small_bf16", [25, 9], 16)
    s = m.shape
    g = torch.Generator(device="cuda").manual_seed(4)
    gains = [[(1 + 0.3 * torch.randn(s.head_dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(s.n_layers)]
             for _ in range(2)]
    m.run([25, 9], q_norm=gains[0], k_norm=gains[1])
    m.ok()
    hq, hkv, d = s.n_q_heads, s.n_kv_heads, s.head_dim
    for b in (0, 1):
        x = fo._f64(m.case.model["embed"])[m.tokens[b]]
        h = fo.rms_norm(x, fo._f64(m.case.model["attn_norm"][0]), s.rms_eps)
        k = (h @ fo._f64(m.case.model["wqkv"][0]).T)[:, hq * d:(hq + hkv) * d].reshape(-1, hkv, d).transpose(1, 0, 2)
        k = fo.rope(fo.rms_norm(k, fo._f64(gains[1][0].cpu()), s.rms_eps), np.arange(k.shape[1]), s.rope_theta)
        # (a relative rounding passes through the norm's scaling unchanged; the row's rms is itself off by at most u)
        _close(cached(m.pool, m.batch["page_table"][b].cpu(), k.shape[1])[0, 0], k, "bf16", "normed K",
               _stored(k, "bf16", True) + 2.0 ** -8 * np.abs(k))
    m.close()


def test_prefill_refusals_and_flags():
    from decodability_aware_token_b200 import ChunkContext, FocusError, _abi
    m = Model("tiny", [20, 7], 16, slots=2, block=16)
    s = m.shape
    with pytest.raises(FocusError) as e:                          # more rows than the context's workspace
        m.run([20, 7], max_rows=33)
    assert e.value.code == _abi.FOCUS_ERR_LIMITS
    with pytest.raises(FocusError) as e:                          # another rotary base
        with ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                          dtype=torch.float32, max_requests=2, max_pages_per_req=m.chunk.limits.max_pages_per_req,
                          rope_theta=5.0) as c:
            m.ctx.prefill(c, torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda(), m.batch,
                          m.free, m.head)
    assert e.value.code == _abi.FOCUS_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        m.ctx.prefill(m.chunk, torch.zeros(1, 3, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda(), m.batch,
                      m.free, m.head)
    torch.cuda.synchronize()
    assert m.batch["prefix_len"].tolist() == [0, 0] and bool(torch.isnan(m.pool).all())   # a refused call changes nothing
    m.tokens[1][2] = s.vocab                                      # a token id out of range, then more tokens than columns
    m.run([20, 7])
    torch.cuda.synchronize()
    assert m.ctx.device_error() == (-5, _abi.FOCUS_DEVERR_TOKEN_ID)
    n = Model("tiny", [20, 7], 16)
    n.ctx.prefill(n.chunk, torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.tensor([3, 4], dtype=torch.int32).cuda(),
                  n.batch, n.free, n.head, max_rows=20)
    torch.cuda.synchronize()
    assert n.ctx.device_error() == (-5, _abi.FOCUS_DEVERR_ROWS)
    m.close(), n.close()


def test_scheduled_prompts_decode_as_if_cached():
    """The scheduler with prompt tokens against the scheduler with the same prompts prefilled before: the same blocks
    in the same number of steps, and the prompts' pages hold the same bits."""
    from decodability_aware_token_b200 import ChunkContext, FocusContext, StepParams
    from decodability_aware_token_b200.scheduler import EffectiveBatchScheduler, FocusEngine, Request
    case = fs.make_case("small_bf16", k_min=1, k_max=4)
    s, w = case.shape, case.work
    model = to_device(case)
    B, S, MP, SLOTS = 16, 16, 10, 4
    g = torch.Generator().manual_seed(9)
    lens = [37, 1, 64, 100, 20, 5]
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in lens]

    def run(with_tokens):
        pool = torch.zeros(60, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.bfloat16, device="cuda")
        free = list(range(60))
        params = StepParams(w.tau, w.k_min, w.k_max, w.conf_threshold, w.alpha)
        with FocusContext(s, model, max_requests=SLOTS, max_block=B, max_keep=B, max_pages_per_req=MP) as ctx, \
                ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                             max_requests=SLOTS, max_pages_per_req=MP, rope_theta=s.rope_theta) as chunk:
            eng = FocusEngine(ctx, params, chunk=chunk, mask_block=B)
            sch = EffectiveBatchScheduler(eng, slots=SLOTS, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads,
                                          head_dim=s.head_dim, max_pages_per_req=MP, kv_pool=pool, free_pages=free,
                                          mask_token=s.vocab - 1, k_max=w.k_max, keep_pages=True)
            for r, toks in enumerate(prompts):
                if with_tokens:
                    sch.submit(Request(r, r, len(toks), [], 1, prompt_tokens=toks))
                    continue
                # one request at a time, chunk by chunk, into pages of its own
                pages = [sch.free.pop() for _ in range(-(-len(toks) // S))]
                view = dict(prefix_len=torch.zeros(1, dtype=torch.int32, device="cuda"), kv_pool=pool,
                            page_table=torch.full((1, MP), -1, dtype=torch.int32, device="cuda"))
                left = torch.tensor(pages, dtype=torch.int32).cuda()
                for p in range(0, len(toks), SLOTS * B):
                    part = torch.tensor([toks[p:p + SLOTS * B]], dtype=torch.int32).cuda()
                    new = torch.tensor([part.shape[1]], dtype=torch.int32).cuda()
                    eng.prefill(view, part, new, left[-(-p // S):])
                assert view["page_table"][0, : len(pages)].tolist() == pages
                sch.submit(Request(r, r, len(toks), pages, 1))
            res = sch.run(max_iterations=500)
            assert ctx.device_error() == (0, 0) and chunk.device_error() == (0, 0)
            return res, pool
    got, pool = run(True)
    want, pool2 = run(False)
    for r, n in enumerate(lens):
        assert [b.tolist() for b in got[r].blocks] == [b.tolist() for b in want[r].blocks]
        assert got[r].steps == want[r].steps and got[r].prefix_len == n + B
        a, b = cached(pool, got[r].pages, n), cached(pool2, want[r].pages, n)
        rms = float(np.sqrt(np.mean(b ** 2)))
        # (a chunk of several requests may split its key walks elsewhere than a request alone: float32 sums in
        # another order, a stored bf16 value one step apart now and then)
        assert float(np.abs(a - b).max()) <= 2e-2 * rms
