"""Prompts in the scheduler, on the CPU: how a call's rows are shared among them, and on how many rows the model runs."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import focus_synth as fs
from prefill_reference import cached, prompt_forward
from test_prefill_cpu import PromptEngine, _run
from test_scheduler_cpu import B, MAX_PAGES, S
from decodability_aware_token_b200 import StepParams
from decodability_aware_token_b200.scheduler import EffectiveBatchScheduler, FocusEngine, Request, share_rows


@pytest.mark.parametrize("step", [1, 8, 32])
def test_rows_of_a_call_are_shared_evenly_in_whole_blocks(step):
    rng = np.random.default_rng(step)
    for _ in range(300):
        left = [int(n) for n in rng.integers(0, rng.choice([2, 40, 3000]), size=rng.integers(1, 18))]
        rows = int(rng.integers(step, 600))
        calls = 0
        while any(left):
            take = share_rows(left, rows, step)
            assert 0 < sum(take) <= rows
            for n, t in zip(left, take):
                assert 0 <= t <= n and (t == n or t % step == 0)
                # nobody gets more than a prompt that goes on after the call, but for the rounding to whole blocks (what
                # one leaves goes in equal parts to the k behind it: less than step (1 + 1/2 + .. + 1/17) = 3.5 step)
                assert all(t <= o + 4 * step or o == m for o, m in zip(take, left))
            spare = rows - sum(take)
            assert spare < step * len(left) or take == left      # what is left over is less than a block each
            left = [n - t for n, t in zip(left, take)]
            calls += 1
            assert calls < 10000
    assert share_rows([1008] + [1] * 15, 1024, 1) == [1008] + [1] * 15
    assert share_rows([5000, 7, 900], 1024, 1) == [509, 7, 508]


def test_the_engine_runs_the_model_on_the_rows_that_hold_tokens():
    """Lengths on the host bound the rows; the scheduler gives them, whatever the longest prompt is."""
    seen = []

    class Context:
        class limits:
            max_requests, max_block = 16, 64

        def prefill(self, chunk, tokens, new_len, batch, pages, head, *, max_rows=None, mask_block=1, stream=None):
            rows = tokens.numel() if max_rows is None else max_rows
            seen.append((rows, int(new_len.sum()), tuple(tokens.shape)))
            batch["prefix_len"] += new_len
    s = fs.make_case("tiny").shape
    eng = FocusEngine(Context(), StepParams(), chunk=SimpleNamespace(limits=SimpleNamespace(max_requests=16)))
    eng.step = lambda view, dense: view["mask"].zero_()
    eng.commit, eng.capacity_check = (lambda view: None), (lambda slots, block: None)
    sch = EffectiveBatchScheduler(eng, slots=16, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                                  max_pages_per_req=200, kv_pool=torch.zeros(400, s.n_layers, 2, s.n_kv_heads, S, s.head_dim),
                                  free_pages=list(range(400)), mask_token=0, k_max=4)
    lens = [700] + [3] * 15
    for r, n in enumerate(lens):
        sch.submit(Request(r, 0, n, [], 1, prompt_tokens=list(range(n))))
    sch.run(max_iterations=50)
    assert [(rows, live) for rows, live, _ in seen] == [(745, 745)] and seen[0][2] == (16, 700)


def test_a_long_prompt_does_not_hold_up_the_requests_that_run():
    """One chunk of prompts per iteration: the running requests step in between, finish when they finish without the
    long prompt, and everybody decodes what it decodes when its prompt was cached before."""
    case = fs.make_case("tiny")
    s, w = case.shape, case.work
    g = torch.Generator().manual_seed(7)
    short = {r: torch.randint(0, s.vocab, (n,), generator=g).tolist() for r, n in ((0, 5), (1, 3))}
    prompts = {**short, 2: torch.randint(0, s.vocab, (40,), generator=g).tolist()}
    kv = {r: prompt_forward(s, case.model, t, 1)[0] for r, t in prompts.items()}

    def run(which):
        pool = torch.zeros(40, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.float64)
        eng = PromptEngine(case, which, kv, 8, 1)
        calls = []
        for what in ("prefill", "step"):
            def note(*a, _f=getattr(eng, what), _w=what, **k):
                calls.append(_w)
                return _f(*a, **k)
            setattr(eng, what, note)
        sch = EffectiveBatchScheduler(eng, slots=3, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads,
                                      head_dim=s.head_dim, max_pages_per_req=MAX_PAGES, kv_pool=pool,
                                      free_pages=list(range(40)), mask_token=s.vocab - 1, k_max=w.k_max, keep_pages=True)
        for r, toks in which.items():
            sch.submit(Request(r, 0 if r < 2 else 1, len(toks), [], 1, prompt_tokens=toks))
        return sch.run(max_iterations=200), calls, sch
    res, calls, sch = run(prompts)
    alone, _, _ = run(short)
    assert calls.count("prefill") == 6                                  # 8 tokens of the short ones, 40 of the long one
    text = " ".join(calls)
    assert "prefill prefill" not in text                                # running requests step between the chunks
    assert [st.prompts for st in sch.stats[:7]] == [0, 1, 1, 1, 1, 0, 0] and all(st.deferred == 0 for st in sch.stats)
    for r in short:
        assert res[r].finished == alone[r].finished and [b.tolist() for b in res[r].blocks] == [b.tolist() for b in alone[r].blocks]
    _, want, _ = _run(case, prompts, kv, False, 8, 1)
    for r in prompts:
        assert [b.tolist() for b in res[r].blocks] == [b.tolist() for b in want[r].blocks]
        np.testing.assert_array_equal(cached(sch.kv_pool, res[r].pages, len(prompts[r])), kv[r])


def test_prompts_that_are_not_cached_yet_wait_behind_the_others():
    """More requests than the row budget runs at once, prompts among them: nothing steps on a prompt that is half done."""
    case = fs.make_case("tiny")
    s, w = case.shape, case.work
    g = torch.Generator().manual_seed(11)
    prompts = {r: torch.randint(0, s.vocab, (n,), generator=g).tolist() for r, n in enumerate((9, 33, 2, 40, 17, 26))}
    kv = {r: prompt_forward(s, case.model, t, 1)[0] for r, t in prompts.items()}
    pool = torch.zeros(60, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.float64)
    eng = PromptEngine(case, prompts, kv, 11, 1)
    sch = EffectiveBatchScheduler(eng, slots=5, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                                  max_pages_per_req=MAX_PAGES, kv_pool=pool, free_pages=list(range(60)),
                                  mask_token=s.vocab - 1, k_max=w.k_max, row_budget=3 * B, keep_pages=True)
    step = eng.step

    def checked(view, dense):
        assert set(view["prefix_len"].tolist()) <= {len(t) + more for t in prompts.values() for more in (0, B)}
        step(view, dense)
    eng.step = checked
    for r, toks in prompts.items():
        sch.submit(Request(r, 0, len(toks), [], 2, prompt_tokens=toks))
    res = sch.run(max_iterations=400)
    _, want, _ = _run(case, prompts, kv, False, 11, 1)
    for r in prompts:
        assert res[r].blocks[0].tolist() == want[r].blocks[0].tolist()
        np.testing.assert_array_equal(cached(pool, res[r].pages, len(prompts[r])), kv[r])


@pytest.mark.parametrize("most", [1, 2])
def test_calls_span_no_more_slots_than_the_chunk_context_takes(most):
    case = fs.make_case("tiny")
    s, w = case.shape, case.work
    g = torch.Generator().manual_seed(5)
    prompts = {r: torch.randint(0, s.vocab, (n,), generator=g).tolist() for r, n in enumerate((9, 21, 0, 14, 30))}
    none = np.zeros((s.n_layers, 2, s.n_kv_heads, 0, s.head_dim))
    kv = {r: prompt_forward(s, case.model, t, 1)[0] if t else none for r, t in prompts.items()}
    eng = PromptEngine(case, prompts, kv, 16, 1)
    eng.prefill_requests = lambda: most
    prefill = eng.prefill

    def checked(view, tokens, new_len, pages):
        assert 1 <= len(new_len) == tokens.shape[0] == view["prefix_len"].shape[0] <= most
        prefill(view, tokens, new_len, pages)
    eng.prefill = checked
    pool = torch.zeros(60, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.float64)
    sch = EffectiveBatchScheduler(eng, slots=5, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                                  max_pages_per_req=MAX_PAGES, kv_pool=pool, free_pages=list(range(60)),
                                  mask_token=s.vocab - 1, k_max=w.k_max, keep_pages=True)
    for r, toks in prompts.items():
        sch.submit(Request(r, 0, len(toks), [], 1, prompt_tokens=toks))
    res = sch.run(max_iterations=300)
    for r in prompts:
        np.testing.assert_array_equal(cached(pool, res[r].pages, len(prompts[r])), kv[r])


def test_the_engine_refuses_a_chunk_context_with_other_page_tables():
    NS = SimpleNamespace
    ctx = NS(limits=NS(max_requests=4, max_block=64, max_keep=64, max_pages_per_req=9))
    eng = lambda pages, n=4: FocusEngine(ctx, StepParams(), chunk=NS(limits=NS(max_requests=n, max_pages_per_req=pages)))
    eng(9).capacity_check(4, 16)
    assert eng(9, 3).prefill_requests() == 3
    with pytest.raises(ValueError):
        eng(8).capacity_check(4, 16)
