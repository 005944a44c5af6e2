"""What focus_prefill stores in the first layer, rounding by rounding (bf16): the normed embedding is rounded to bf16, the
projection accumulates in float32, keys are rotated from there and rounded once, values are rounded once.

Bound per element, with h the rounded row, w a weight row, u = 2^-8 half a step and E = 2^-24: the store u |out|; the
float32 sum D E sum |h w|, a turn adds 8 E (angles and products); float32 norms may round an element of h the other way
where it lies within 4 E of a tie, which adds a step of h there."""
import numpy as np
import pytest
import torch

import focus_synth as fs
from oracle import focus_oracle as fo
from prefill_reference import cached
from test_gpu_prefill import Model

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def _pair(x):
    lo, hi = np.split(x, 2, axis=-1)
    return np.concatenate([lo + hi, lo + hi], axis=-1)


@pytest.mark.parametrize("name,lens,kw", [
    ("small_bf16", [1], {}), ("small_bf16", [60, 3, 90], {}), ("small_bf16", [300], {}),             # each GEMM kernel
    ("small_bf16", [100, 99, 101, 80, 100], dict(max_rows=500)), ("small_bf16_g4", [37, 50], {}),
    ("wide_bf16", [200, 140], {}), ("small_bf16", [20, 20], dict(splits=[[7, 0], [13, 20]])),
])
def test_first_layer_keys_and_values_are_rounded_once(name, lens, kw):
    kw = dict(kw)
    m = Model(name, lens, 16)
    s, hq, hkv, d = m.shape, m.shape.n_q_heads, m.shape.n_kv_heads, m.shape.head_dim
    for new in kw.pop("splits", None) or [lens]:
        m.run(new, **kw)
    m.ok()
    w = fo._f64(m.case.model["wqkv"][0])[hq * d:]
    for b, n in enumerate(lens):
        x = fo._f64(m.case.model["embed"])[m.tokens[b]]
        h64 = fo.rms_norm(x, fo._f64(m.case.model["attn_norm"][0]), s.rms_eps)
        h, either = _bf16(h64), np.abs(_bf16(h64 * (1 + 4 * E)) - _bf16(h64 * (1 - 4 * E)))
        out, mag, slack = h @ w.T, np.abs(h) @ np.abs(w).T, either @ np.abs(w).T
        heads = lambda a: a.reshape(n, 2, hkv, d).transpose(1, 2, 0, 3)
        out, mag, slack = heads(out), heads(mag), heads(slack)
        k = fo.rope(out[0], np.arange(n), s.rope_theta)
        got = cached(m.pool, m.batch["page_table"][b].cpu(), n)[0]
        D = s.hidden
        for what, g, want, bound in (("V", got[1], out[1], D * E * mag[1] + slack[1]),
                                     ("K", got[0], k, _pair((D + 8) * E * mag[0] + slack[0]))):
            over = np.abs(g - want) - (U * np.abs(want) + 1.01 * bound)
            assert over.max() <= 0, (what, b, float(over.max()), float((over > 0).mean()))
    m.close()


def test_page_tables_beyond_the_contexts_angles_are_rotated_by_the_operator():
    """A chunk context of longer page tables than the model's context: the same keys, up to one more rounding."""
    from decodability_aware_token_b200 import ChunkContext
    lens = [40, 9]
    a, b = Model("small_bf16", lens, 16), Model("small_bf16", lens, 16)
    s, mp = a.shape, a.chunk.limits.max_pages_per_req
    wide = 5 * mp + 16                                            # 16 x (5 mp + 16) > 64 mp + 64
    b.chunk.close()
    b.chunk = ChunkContext(n_layers=s.n_layers, n_q_heads=s.n_q_heads, n_kv_heads=s.n_kv_heads, head_dim=s.head_dim,
                           max_requests=2, max_pages_per_req=wide, rope_theta=s.rope_theta)
    b.batch["page_table"] = torch.full((2, wide), -1, dtype=torch.int32, device="cuda")
    a.run(lens), b.run(lens)
    a.ok(), b.ok()
    x, y = (cached(m.pool, m.batch["page_table"][0].cpu(), 40) for m in (a, b))
    assert np.array_equal(x[0, 1], y[0, 1]) and not np.array_equal(x[0, 0], y[0, 0])
    r = np.sqrt(_pair(x[0, 0] ** 2))
    assert (np.abs(x[0, 0] - y[0, 0]) <= (2 + np.sqrt(2)) * U * r + 1e-6).all()
    a.close(), b.close()
