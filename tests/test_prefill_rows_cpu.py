"""Prompts in the scheduler, on the CPU: how a call's rows are shared among them, and on how many rows the model runs."""
import numpy as np
import pytest
import torch

import focus_synth as fs
from test_scheduler_cpu import B, S
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
    eng = FocusEngine(Context(), StepParams(), chunk=object())
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
