"""Prompts on exactly as many rows as they have tokens, on the GPU, against the float64 forward (tolerances of
test_gpu_prefill.py): one row, row counts around the GEMMs' tiles, and one long prompt among short ones."""
import pytest
import torch

from prefill_reference import cached, prompt_forward
from test_gpu_prefill import Model, _close, _stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,lens", [
    ("small_bf16", [1]), ("small_bf16", [2]), ("small_bf16", [31, 2]), ("small_bf16", [0, 127]), ("small_bf16", [120, 9]),
    ("small_bf16", [255]), ("small_bf16", [250, 7]), ("small_bf16", [150, 3, 1, 2, 3, 1, 2, 3]), ("tiny", [1]), ("tiny", [63, 2]),
])
def test_prefill_on_exactly_the_rows_that_hold_tokens(name, lens):
    m = Model(name, lens, 16)
    plan = m.run(lens, max_rows=sum(lens))
    m.ok()
    assert plan.row_req.shape[0] == sum(lens) and m.batch["prefix_len"].tolist() == lens
    table = m.batch["page_table"].cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kv, _ = prompt_forward(m.shape, m.case.model, m.tokens[b], 1)
        got = cached(m.pool, table[b], n)
        for l in range(m.shape.n_layers):
            for i, what in enumerate(("K", "V")):
                _close(got[l, i], kv[l, i], m.shape.dtype, f"{what} of request {b}, layer {l}",
                       _stored(kv[l, i], m.shape.dtype, what == "K"))
    m.close()


def test_the_engine_takes_lengths_on_the_host():
    from decodability_aware_token_b200 import StepParams
    from decodability_aware_token_b200.scheduler import FocusEngine
    lens = [70, 5, 0, 31]
    pools = []
    for where in ("cpu", "cuda"):
        m = Model("small_bf16", lens, 16)
        eng = FocusEngine(m.ctx, StepParams(), chunk=m.chunk)
        tok = torch.zeros(4, 70, dtype=torch.int32)
        for b, t in enumerate(m.tokens):
            tok[b, : len(t)] = torch.tensor(t, dtype=torch.int32)
        eng.prefill(m.batch, tok.to(where), torch.tensor(lens, dtype=torch.int32).to(where), m.free.to(where))
        m.ok()
        assert m.batch["prefix_len"].tolist() == lens
        pools.append((m.pool.nan_to_num(nan=9.0).float(), m.batch["page_table"].clone()))
        m.close()
    (a, ta), (b, tb) = pools
    assert torch.equal(ta, tb)
    # (other row counts take other GEMM kernels: sums in another order)
    assert float((a - b).abs().max()) <= 2e-2 * float(a.square().mean().sqrt())
