"""Requests that bring their prompt's tokens, on the CPU: the scheduler runs the prompts through the engine in chunks
at admission, in their own pages, and every request then decodes what it decodes when its prompt's keys and values
were in the pool from the start."""
import numpy as np
import pytest
import torch

import focus_synth as fs
from prefill_reference import cached, prompt_forward
from test_scheduler_cpu import B, MAX_PAGES, S, OracleEngine
from decodability_aware_token_b200.scheduler import EffectiveBatchScheduler, Request


class PromptEngine(OracleEngine):
    """The oracle engine plus a prefill that writes precomputed keys and values the way the library does: pages from
    the list in request order, positions prefix_len .. prefix_len + new_len - 1."""

    def __init__(self, case, prompts, kv, rows, mask_block):
        super().__init__(case)
        self.prompts, self.kv, self.rows, self.mask_block = prompts, kv, rows, mask_block
        self.chunks = []

    def prefill_rows(self):
        return self.rows

    def prefill(self, view, tokens, new_len, pages):
        pages, n_new = pages.tolist(), new_len.tolist()
        assert sum(n_new) <= self.rows and tokens.shape[1] >= max(n_new)
        for b, n in enumerate(n_new):
            if n == 0:
                continue
            p = int(view["prefix_len"][b])
            rid = next(r for r, t in self.prompts.items() if t[p:p + n] == tokens[b, :n].tolist())
            assert p % self.mask_block == 0 and (n % self.mask_block == 0 or p + n == len(self.prompts[rid]))
            for i in range(-(-p // S), -(-(p + n) // S)):
                assert int(view["page_table"][b, i]) == pages[0]
                pages.pop(0)
            for j in range(p, p + n):
                view["kv_pool"][int(view["page_table"][b, j // S]), :, :, :, j % S] = torch.as_tensor(self.kv[rid][:, :, :, j])
            view["prefix_len"][b] = p + n
            self.chunks.append((rid, p, n))
        assert not pages


def _run(case, prompts, kv, with_tokens, rows, mask_block, slots=3):
    s, w = case.shape, case.work
    n_pages = 40
    pool = torch.zeros(n_pages, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.float64)
    free = list(range(n_pages))[::-1]
    eng = PromptEngine(case, prompts, kv, rows, mask_block)
    sch = EffectiveBatchScheduler(eng, slots=slots, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads,
                                  head_dim=s.head_dim, max_pages_per_req=MAX_PAGES, kv_pool=pool, free_pages=free,
                                  mask_token=s.vocab - 1, k_max=w.k_max, keep_pages=True)
    for rid, toks in prompts.items():
        P = len(toks)
        if with_tokens:
            sch.submit(Request(rid, rid // 2, P, [], 1, prompt_tokens=toks))
        else:
            pages = [sch.free.pop() for _ in range(-(-P // S))]
            for j in range(P):
                pool[pages[j // S], :, :, :, j % S] = torch.as_tensor(kv[rid][:, :, :, j])
            sch.submit(Request(rid, rid // 2, P, pages, 1))
    res = sch.run(max_iterations=200)
    return eng, res, pool


@pytest.mark.parametrize("rows,mask_block", [(64, 1), (7, 1), (64, 8), (16, 8)])
def test_prompts_are_prefilled_in_chunks_and_decode_as_if_cached(rows, mask_block):
    case = fs.make_case("tiny")
    g = torch.Generator().manual_seed(3)
    prompts = {r: torch.randint(0, case.shape.vocab, (n,), generator=g).tolist() for r, n in enumerate((17, 1, 30, 0, 21))}
    kv = {r: prompt_forward(case.shape, case.model, t, mask_block)[0] if t else np.zeros((case.shape.n_layers, 2, case.shape.n_kv_heads, 0, case.shape.head_dim))
          for r, t in prompts.items()}
    eng, res, pool = _run(case, prompts, kv, True, rows, mask_block)
    _, want, _ = _run(case, prompts, kv, False, rows, mask_block)
    assert sorted(res) == sorted(want) == list(prompts)
    for r in prompts:
        assert [b.tolist() for b in res[r].blocks] == [b.tolist() for b in want[r].blocks]
        assert res[r].prefix_len == len(prompts[r]) + B
        np.testing.assert_array_equal(cached(pool, res[r].pages, len(prompts[r])), kv[r])
        chunks = [(p, n) for rid, p, n in eng.chunks if rid == r]
        assert sum(n for _, n in chunks) == len(prompts[r])
    assert (len(eng.chunks) > 4) == (rows < 64)


def test_submit_refuses_prompts_the_engine_cannot_take():
    case = fs.make_case("tiny")
    s, w = case.shape, case.work
    pool = torch.zeros(8, s.n_layers, 2, s.n_kv_heads, S, s.head_dim, dtype=torch.float64)

    def make(engine):
        return EffectiveBatchScheduler(engine, slots=2, block=B, n_layers=s.n_layers, n_kv_heads=s.n_kv_heads,
                                       head_dim=s.head_dim, max_pages_per_req=MAX_PAGES, kv_pool=pool,
                                       free_pages=list(range(8)), mask_token=s.vocab - 1, k_max=w.k_max)
    with pytest.raises(ValueError):
        make(OracleEngine(case)).submit(Request(0, 0, 2, [], 1, prompt_tokens=[1, 2]))      # no prefill
    eng = PromptEngine(case, {}, {}, 16, 1)
    with pytest.raises(ValueError):
        make(eng).submit(Request(0, 0, 3, [], 1, prompt_tokens=[1, 2]))                     # length
    with pytest.raises(ValueError):
        make(eng).submit(Request(0, 0, 2, [1], 1, prompt_tokens=[1, 2]))                    # pages and tokens
    with pytest.raises(ValueError):
        make(PromptEngine(case, {}, {}, 16, 32)).submit(Request(0, 0, 2, [], 1, prompt_tokens=[1, 2]))  # block > rows


def test_one_block_per_chunk_reference_is_the_dense_forward():
    """The float64 reference itself: a mask block as long as the prompt is one bidirectional pass, blocks of one are
    the causal pass, whose rows do not depend on later tokens."""
    case = fs.make_case("tiny")
    toks = torch.randint(0, case.shape.vocab, (9,), generator=torch.Generator().manual_seed(1)).tolist()
    kv, hid = prompt_forward(case.shape, case.model, toks, 1)
    kv2, hid2 = prompt_forward(case.shape, case.model, toks[:6], 1)
    np.testing.assert_allclose(kv[:, :, :, :6], kv2, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(hid[:6], hid2, rtol=1e-12, atol=1e-12)
    full, _ = prompt_forward(case.shape, case.model, toks, 9)
    assert np.abs(full[1:, :, :, 0] - kv[1:, :, :, 0]).max() > 1e-3   # position 0 sees the rest of its block
