"""Chunk operators on the GPU against plain 64-bit implementations: page plan, query/key norm + rotation + cache
write, attention over the paged cache -- at the sizes and masks where they can go wrong, with their device-side
refusals, in graphs, on other streams, and as the run in which they are used.

Tolerances.  u is half a step of the stored type relative to the value: 2^-8 for bf16, 2^-24 for float32.
  norm + rotation: y = x / rms * gain, then y c - y' s.  Float32 work before the one rounding: the sum of d squares
  and the scaling cost (d + 8) 2^-24 relative, the angle's factors 8 2^-24 absolute (the reduced angle is rounded
  once, sincospif is good to 2 units), so |error| <= u |out| + (d + 24) 2^-24 (|y| + |y'|).
  attention: with weights w_j (sum 1), A = sum w_j |V_j| and B the largest sum_i |q_i k_i| scale of a row: scores are
  off by at most (d + 6) 2^-24 B, which moves each weight by twice that relative (itself and the denominator);
  sums over n keys add (n / 16 + 64) 2^-24 (chains of at most n / 16 terms before they are joined, and the
  joins); float32 weights are good to 2^-22.  bf16 weights are rounded before the product with V (2^-8 each, the
  denominator is not).
  |error| <= u |out| + A (2 (d + 6) 2^-24 B + (n / 16 + 64) 2^-24 + 2^-22 + [bf16] 2^-8).
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: torch.finfo(BF).eps / 2, F32: torch.finfo(F32).eps / 2}
E = 2.0 ** -24


def _ctx(hq=4, hkv=2, d=128, dtype=BF, n=64, pages=64, layers=2, theta=10000.0):
    from decodability_aware_token_b200 import ChunkContext
    return ChunkContext(n_layers=layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, dtype=dtype, max_requests=n,
                        max_pages_per_req=pages, rope_theta=theta, device="cuda:0")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------------------ plan
def _plan_plain(prefix, new, table, free, head, S, n_pages, T, max_pages):
    """Request by request, as the header states it; returns the outputs and the error bits."""
    table = [list(r) for r in table]
    bits = 0
    if not 0 <= head <= len(free):
        bits |= 2
        avail = 0
    else:
        avail = len(free) - head
    offs, kv, req, pos, slot, asked, need_sum, at = [0], [], [], [], [], 0, 0, head
    ok_page = lambda p: 0 <= p < n_pages
    for b, (p, n) in enumerate(zip(prefix, new)):
        rows = 0
        if p < 0 or n < 0 or p + n > max_pages * S:
            bits |= 4
        else:
            asked += n
            if n == 0 or asked <= T:
                have = _ceil(p, S)
                need = _ceil(p + n, S) - have
                need_sum += need
                if need == 0 or need_sum <= avail:
                    rows = n
                    for i in range(need):
                        if not ok_page(free[at]):
                            bits |= 2
                        table[b][have + i] = free[at] if ok_page(free[at]) else -1
                        at += 1
        for i in range(rows):
            pg = table[b][(p + i) // S]
            if not ok_page(pg):
                bits |= 2
            req.append(b)
            pos.append(p + i)
            slot.append(pg * S + (p + i) % S if ok_page(pg) else -1)
        offs.append(len(req))
        kv.append(p + rows)
    pad = [-1] * (T - len(req))
    return [offs, kv, req + pad, pos + pad, slot + pad, table, [at]], bits


def _plan_case(rng, N, S, T, max_pages, spare, max_new, max_prefix, head=0):
    prefix = [rng.randint(0, min(max_prefix, max_pages * S)) for _ in range(N)]
    new = [rng.randint(0, max(0, min(max_new, max_pages * S - p))) for p in prefix]
    have = [_ceil(p, S) for p in prefix]
    want = sum(_ceil(p + n, S) - h for p, n, h in zip(prefix, new, have))
    n_free = head + int(want * spare)
    n_pages = sum(have) + n_free + 2
    ids = rng.sample(range(n_pages), n_pages)
    table, at = [], 0
    for h in have:
        table.append(ids[at:at + h] + [-1] * (max_pages - h))
        at += h
    return prefix, new, table, ids[at:at + n_free], n_pages


def _run_plan(ctx, prefix, new, table, free, head, S, n_pages, T, alias=False):
    t, h = _i32(table).reshape(len(prefix), ctx.limits.max_pages_per_req), _i32([head])
    out = ctx.alloc_plan(len(prefix), T)
    if alias:
        out.free_next = h
    ctx.plan(_i32(prefix), _i32(new), t, _i32(free), h, page_size=S, n_pages=n_pages, out=out)
    torch.cuda.synchronize()
    return [x.tolist() for x in (out.row_offsets, out.kv_len, out.row_req, out.row_pos, out.row_slot, t, out.free_next)]


@pytest.mark.parametrize("N,S,T,spare,max_new,max_prefix", [
    (1, 16, 1, 1.0, 1, 40), (1, 64, 5, 1.0, 9, 0), (5, 1, 64, 1.0, 12, 9), (7, 7, 300, 1.0, 50, 30),
    (32, 64, 32, 1.0, 1, 200), (33, 16, 4000, 0.6, 200, 100), (255, 32, 9000, 1.0, 64, 200),
    (256, 16, 3000, 1.0, 40, 100), (257, 16, 5000, 0.4, 40, 100), (700, 16, 20000, 0.9, 60, 50), (40, 16, 0, 1.0, 3, 9),
])
def test_plan_matches_the_rules(N, S, T, spare, max_new, max_prefix):
    rng = random.Random(N * 1000 + S)
    for head in (0, 3):
        mp = _ceil(max_prefix + max_new, S) + 1
        with _ctx(n=N, pages=mp) as ctx:
            p, n, table, free, n_pages = _plan_case(rng, N, S, T, mp, spare, max_new, max_prefix, head)
            want, bits = _plan_plain(p, n, table, free, head, S, n_pages, T, mp)
            got = _run_plan(ctx, p, n, table, free, head, S, n_pages, T, alias=head > 0)
            assert got == want
            assert ctx.device_error() == (0, 0) and bits == 0


def test_plan_flags_bad_input_and_goes_on():
    S, mp, T = 16, 4, 64
    with _ctx(n=8, pages=mp) as ctx:
        cases = [
            ([5, -1, 3], [4, 2, 6], [[0, 9, 9, 9], [1, 9, 9, 9], [2, 9, 9, 9]], [7, 8], 0),      # negative prefix
            ([5, 3, 3], [4, -2, 60], [[0, 9, 9, 9], [1, 9, 9, 9], [2, 9, 9, 9]], [7, 8, 10, 11], 0),  # negative new
            ([60, 3], [5, 1], [[0, 1, 2, 3], [4, 9, 9, 9]], [7, 8], 0),                           # beyond the table
            ([16, 3], [16, 1], [[0, 9, 9, 9], [1, 9, 9, 9]], [99, 8], 0),                         # bad free page
            ([3, 3], [2, 2], [[-1, 9, 9, 9], [500, 9, 9, 9]], [7], 0),                            # bad table entries
            ([16, 3], [16, 1], [[0, 9, 9, 9], [1, 9, 9, 9]], [7, 8], 3),                          # head past the list
            ([16, 3], [16, 1], [[0, 9, 9, 9], [1, 9, 9, 9]], [7, 8], -1),                         # negative head
        ]
        for p, n, table, free, head in cases:
            want, bits = _plan_plain(p, n, table, free, head, S, 20, T, mp)
            assert bits
            assert _run_plan(ctx, p, n, table, free, head, S, 20, T) == want
            assert ctx.device_error() == (-5, bits)
            assert ctx.device_error() == (0, 0)


def test_plan_of_no_requests_and_in_a_graph():
    S, mp, T, N = 16, 8, 40, 6
    with _ctx(n=N, pages=mp) as ctx:
        assert _run_plan(ctx, [], [], [], [4], 1, S, 5, 3) == [[0], [], [-1] * 3, [-1] * 3, [-1] * 3, [], [1]]
        # a captured plan sees the lengths of each replay; the free list runs on through free_head
        pre, new = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
        table = torch.full((N, mp), -1, dtype=torch.int32, device="cuda")
        free, head = torch.arange(50, dtype=torch.int32, device="cuda").flip(0), _i32([0])
        out = ctx.alloc_plan(N, T)
        out.free_next = head
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.plan(pre, new, table, free, head, page_size=S, n_pages=50, out=out)
        rng = random.Random(5)
        hp, ht, hh = [0] * N, [[-1] * mp for _ in range(N)], 0
        for _ in range(4):
            hn = [rng.randint(0, 12) for _ in range(N)]
            new.copy_(_i32(hn))
            g.replay()
            torch.cuda.synchronize()
            want, _ = _plan_plain(hp, hn, ht, free.tolist(), hh, S, 50, T, mp)
            got = [x.tolist() for x in (out.row_offsets, out.kv_len, out.row_req, out.row_pos, out.row_slot, table, head)]
            assert got == want
            hp, ht, hh = want[1], want[5], want[6][0]
            pre.copy_(out.kv_len)
        assert ctx.device_error() == (0, 0)


# ------------------------------------------------------------------------------- norm, rotation, cache write
def _turn64(x, gain, pos, theta, eps):
    """(out, |y| + |partner|) of x [rows, heads, d] in float64."""
    x = x.double()
    d = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    ang = pos.double()[:, None] * theta ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    mag = (lo.abs() + hi.abs()).repeat(1, 1, 2)
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1), mag


def _check_turn(got, want, mag, dt):
    d = want.shape[-1]
    err = (got.double() - want).abs()
    tol = U[dt] * want.abs() + (d + 24) * E * mag
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("dt,hq,hkv,d,S,T,norms,start", [
    (BF, 4, 2, 128, 16, 1, "qk", 0), (BF, 16, 8, 128, 64, 33, "qk", 1000), (BF, 32, 8, 128, 32, 130, "", 65530),
    (BF, 6, 2, 128, 16, 77, "q", 1 << 20), (BF, 5, 1, 128, 64, 19, "k", 3), (BF, 1, 1, 128, 7, 9, "qk", 0),
    (F32, 4, 4, 64, 16, 50, "qk", 500), (F32, 4, 4, 64, 1, 3, "", 9), (F32, 12, 3, 128, 24, 31, "qk", 70000),
    (F32, 2, 1, 64, 16, 2000, "qk", 0),
])
def test_norm_rotation_and_cache_write(dt, hq, hkv, d, S, T, norms, start):
    g = torch.Generator(device="cuda").manual_seed(hq * 1000 + T)
    n_pages, L, layer, eps = _ceil(T, S) + 2, 3, 1, 1e-6
    wide = torch.randn(T, hq + 2 * hkv + 1, d, generator=g, device="cuda").mul_(3).to(dt)
    wide[T // 2, 0] *= 1e-4                                      # a tiny head: eps matters
    q, k, v = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:hq + 2 * hkv]
    pos = (torch.arange(T, device="cuda") + start).to(torch.int32)
    slot = torch.randperm(n_pages * S, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 4:
        pos[1], slot[3] = -1, -1                                 # a row to skip, a row not to store
    gq = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if "q" in norms else None
    gk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if "k" in norms else None
    pool = torch.randn(n_pages, L, 2, hkv, S, d, generator=g, device="cuda").to(dt)
    before, out0 = pool.clone(), torch.full((T, hq, d), 7.0, dtype=dt, device="cuda")
    with _ctx(hq, hkv, d, dt, layers=L, theta=50000.0) as ctx:
        out = ctx.qk_norm_rope(q, k, v, pool, layer, pos, slot, q_norm=gq, k_norm=gk, eps=eps, out=out0)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        live = pos >= 0
        _check_turn(out[live], *[x[live] for x in _turn64(q, gq, pos, 50000.0, eps)], dt)
        assert bool((out[~live] == 7).all())
        st = live & (slot >= 0)
        pg, at = (slot[st] // S).long(), (slot[st] % S).long()
        _check_turn(pool[pg, layer, 0, :, at], *[x[st] for x in _turn64(k, gk, pos, 50000.0, eps)], dt)
        assert torch.equal(pool[pg, layer, 1, :, at], v[st])
        pool[pg, layer, :, :, at] = before[pg, layer, :, :, at]
        assert torch.equal(pool, before)                         # nothing else was written
        # in place, on another stream
        q2, s = q.contiguous(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ctx.qk_norm_rope(q2, k, v, pool, layer, pos, slot, q_norm=gq, k_norm=gk, eps=eps, out=q2, stream=s)
        s.synchronize()
        assert torch.equal(q2[live], out[live]) and torch.equal(q2[~live], q[~live])


def test_cache_write_refuses_bad_slots_and_keeps_rows_apart():
    with _ctx(2, 1, 128, BF, layers=1) as ctx:
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(4, 4, 128, generator=g, device="cuda").to(BF)
        x[1] = float("nan")                                      # one row's NaN stays in that row
        x[2, 1] = float("inf")
        pool = torch.zeros(2, 1, 2, 1, 16, 128, dtype=BF, device="cuda")
        gain = torch.ones(128, dtype=BF, device="cuda")
        slot = _i32([0, 1, 32, 2147483647])                      # two pages of 16: 32 is past the pool
        out = ctx.qk_norm_rope(x[:, :2], x[:, 2:3], x[:, 3:], pool, 0, _i32([0, 1, 2, 3]), slot, q_norm=gain, k_norm=gain)
        torch.cuda.synchronize()
        assert ctx.device_error() == (-5, 2)
        assert bool(torch.isfinite(out[[0, 3]]).all()) and bool(torch.isfinite(out[2, 0]).all())
        assert bool(torch.isnan(out[1]).all())
        assert bool((pool[0, 0, :, 0, 2:] == 0).all()) and bool((pool[1] == 0).all())
        empty = ctx.qk_norm_rope(x[:0, :2], x[:0, 2:3], x[:0, 3:], pool, 0, _i32([]), _i32([]))
        assert empty.shape == (0, 2, 128)


# ------------------------------------------------------------------------------------------------ attention
class Batch:
    """A paged batch: requests (rows n, cached keys kv); page tails and unused pages hold NaN."""

    def __init__(self, reqs, hq, hkv, d, dt, S, seed=0, layers=2, pad=0, gain=2.0, slack=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.reqs, self.hq, self.hkv, self.d, self.dt, self.S, self.layers = reqs, hq, hkv, d, dt, S, layers
        need = [_ceil(kv, S) for _, kv in reqs]
        self.max_pages = max(need + [0]) + slack
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        self.pool = torch.full((n_pages, layers, 2, hkv, S, d), float("nan"), dtype=dt, device="cuda")
        self.table = torch.full((len(reqs), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, (n, kv) in enumerate(reqs):
            pages = order[at:at + need[b]]
            at += need[b]
            self.table[b, : need[b]] = torch.tensor(pages, dtype=torch.int32)
            for i, p in enumerate(pages):
                m = min(S, kv - i * S)
                self.pool[p, :, :, :, :m] = torch.randn(layers, 2, hkv, m, d, generator=g, device="cuda").to(dt)
        self.table = self.table.cuda()
        self.offs = [0]
        for n, _ in reqs:
            self.offs.append(self.offs[-1] + n)
        self.T = self.offs[-1] + pad
        self.q = torch.randn(self.T, hq, d, generator=g, device="cuda").mul_(gain).to(dt)
        self.row_offsets, self.kv_len = _i32(self.offs), _i32([kv for _, kv in reqs])

    def run(self, ctx, mask_block=1, out=None, layer=1, **kw):
        return ctx.attention(self.q, self.pool, layer, self.row_offsets, self.kv_len, self.table, mask_block=mask_block,
                             out=out, **kw)

    def check(self, out, mask_block=1, layer=1, scale=None, skip=(), missing=None):
        """`missing`: {request: set of key positions whose page is not mapped}"""
        scale = scale or 1 / math.sqrt(self.d)
        G = self.hq // self.hkv
        for b, (n, kv) in enumerate(self.reqs):
            if b in skip or n == 0:
                continue
            r0 = self.offs[b]
            got = out[r0:r0 + n].double()
            pos = torch.arange(kv - n, kv, device="cuda")
            keys = torch.arange(kv, device="cuda")
            seen = (keys[None] < ((pos // mask_block + 1) * mask_block)[:, None]) & (pos >= 0)[:, None]
            if missing and b in missing:
                seen[:, sorted(missing[b])] = False
            if kv == 0:
                assert bool((got == 0).all())
                continue
            pages = self.table[b, : _ceil(kv, self.S)].long().clamp(min=0, max=self.pool.shape[0] - 1)
            k, v = [torch.nan_to_num(self.pool[pages, layer, i].double()).transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :kv]
                    for i in (0, 1)]
            q = self.q[r0:r0 + n].double().reshape(n, self.hkv, G, self.d).permute(1, 2, 0, 3)
            sc = (q @ k[:, None].transpose(-1, -2)) * scale
            big = ((q.abs() @ k[:, None].abs().transpose(-1, -2)) * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
            sc = sc.masked_fill(~seen, -torch.inf)
            m = sc.amax(-1, keepdim=True)
            w = torch.exp(sc - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
            want, A = w @ v[:, None], w @ v[:, None].abs()
            tol = U[self.dt] * want.abs() + A * (2 * (self.d + 6) * E * big + (kv / 16 + 64) * E + 2.0 ** -22 +
                                                 (2.0 ** -8 if self.dt == BF else 0))
            err = (got.reshape(n, self.hkv, G, self.d).permute(1, 2, 0, 3) - want).abs()
            assert bool((err <= tol).all()), (b, n, kv, float((err - tol).max()))


HEADS = [(BF, 4, 4, 128), (BF, 16, 8, 128), (BF, 32, 8, 128), (BF, 6, 2, 128), (BF, 8, 1, 128), (BF, 17, 1, 128),
         (BF, 64, 1, 128), (BF, 20, 4, 128), (F32, 4, 4, 64), (F32, 8, 2, 64), (F32, 6, 2, 128), (F32, 16, 1, 128)]


@pytest.mark.parametrize("dt,hq,hkv,d", HEADS)
@pytest.mark.parametrize("mask_block", [1, 32, 1 << 30])
def test_attention_head_layouts(dt, hq, hkv, d, mask_block):
    # single tokens, short and long chunks, a whole prompt, kv at and around the block and page edges
    reqs = [(1, 1), (1, 64), (1, 65), (2, 2), (1, 200), (3, 130), (17, 17), (130, 130), (65, 129), (1, 63), (40, 300)]
    b = Batch(reqs, hq, hkv, d, dt, 16, seed=hq, pad=3)
    with _ctx(hq, hkv, d, dt, n=len(reqs), pages=b.max_pages) as ctx:
        out = torch.full_like(b.q, 5.0)
        b.run(ctx, mask_block, out)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        b.check(out, mask_block)
        assert bool((out[b.offs[-1]:] == 5).all())               # rows behind the last request


@pytest.mark.parametrize("dt,S", [(BF, 16), (BF, 32), (BF, 64), (F32, 1), (F32, 7), (F32, 16), (F32, 100)])
@pytest.mark.parametrize("mask_block", [1, 7, 64, 100])
def test_attention_pages_and_masks(dt, S, mask_block):
    d = 128 if dt == BF else 64
    rng = random.Random(S * 7 + mask_block)
    reqs = [(n, n + rng.randint(0, 150)) for n in [rng.choice([1, 1, 2, 5, 16, 33, 64, 100, 129]) for _ in range(14)]]
    b = Batch(reqs, 8, 2, d, dt, S, seed=S)
    with _ctx(8, 2, d, dt, n=len(reqs), pages=b.max_pages) as ctx:
        out = b.run(ctx, mask_block, max_new=max(n for n, _ in reqs))
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        b.check(out, mask_block)
        b.check(b.run(ctx, mask_block, scale=0.3), mask_block, scale=0.3)
        assert torch.equal(b.run(ctx, mask_block), out)          # the bound on new tokens does not change results


@pytest.mark.parametrize("dt,hq,hkv,d", [(BF, 4, 1, 128), (BF, 1, 1, 128), (F32, 4, 1, 64)])
def test_attention_long_walk_split_over_many_ctas(dt, hq, hkv, d):
    """One or two units whose key walk is shared by (nearly) every CTA; rows with very large scores, where the
    running maximum is raised again and again."""
    kv = 40000 if dt == BF else 9000
    for n in (1, 3, 40):
        b = Batch([(n, kv + n)], hq, hkv, d, dt, 64, seed=n, layers=1, gain=4.0)
        with _ctx(hq, hkv, d, dt, n=1, pages=b.max_pages, layers=1) as ctx:
            out = b.run(ctx, layer=0)
            torch.cuda.synchronize()
            assert ctx.device_error() == (0, 0)
            b.check(out, layer=0)
    b = Batch([(5, 3000), (130, 2500)], hq, hkv, d, dt, 64, seed=9, layers=1, gain=40.0)
    b.pool[..., 0] = torch.linspace(-1, 3, b.pool.shape[-2], device="cuda").to(dt)
    with _ctx(hq, hkv, d, dt, n=2, pages=b.max_pages, layers=1) as ctx:
        b.check(b.run(ctx, layer=0), layer=0)


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
def test_attention_empty_rows(dt, d):
    """Rows before position 0 and requests without keys or rows: zeros, nothing or no change."""
    reqs = [(5, 3), (1, 0), (40, 0), (0, 17), (70, 20), (0, 0), (1, 9)]
    b = Batch(reqs, 8, 2, d, dt, 16, seed=3, pad=2)
    with _ctx(8, 2, d, dt, n=len(reqs), pages=b.max_pages) as ctx:
        out = torch.full_like(b.q, 5.0)
        b.run(ctx, 1, out)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0)
        b.check(out)
        assert bool((out[:2] == 0).all()) and bool((out[5:46] == 0).all()) and bool((out[46:96] == 0).all())
        assert bool((out[b.offs[-1]:] == 5).all())
        # no request has rows; no pages at all
        none = Batch([(0, 5), (0, 0)], 8, 2, d, dt, 16, pad=4)
        keep = torch.full_like(none.q, 5.0)
        none.run(ctx2 := _ctx(8, 2, d, dt, n=2, pages=none.max_pages), 1, keep)
        assert bool((keep == 5).all())
        empty_pool = torch.zeros(0, 2, 2, 2, 16, d, dtype=dt, device="cuda")
        o = ctx2.attention(none.q[:2], empty_pool, 0, _i32([0, 1, 2]), _i32([0, 0]), none.table)
        assert bool((o == 0).all()) and ctx2.device_error() == (0, 0)
        assert ctx2.attention(none.q[:0], empty_pool, 0, _i32([0]), _i32([]), none.table[:0]).shape == (0, 8, d)
        ctx2.close()


@pytest.mark.parametrize("dt,d,S", [(BF, 128, 16), (BF, 128, 64), (F32, 64, 16)])
def test_attention_flags_bad_pages_rows_and_lengths(dt, d, S):
    reqs = [(1, 100), (70, 200), (1, 5), (3, 40), (50, 90)]
    b = Batch(reqs, 4, 2, d, dt, S, seed=4)
    b.table[0, 1] = -1
    b.table[1, 2] = b.pool.shape[0]
    missing = {0: set(range(S, min(100, 2 * S))), 1: set(range(2 * S, min(200, 3 * S)))}
    with _ctx(4, 2, d, dt, n=5, pages=b.max_pages) as ctx:
        out = b.run(ctx)
        torch.cuda.synchronize()
        assert ctx.device_error() == (-5, 2)
        b.check(out, missing=missing)
        # all pages bad: no key is left, the rows are zero
        table = b.table.clone()
        table[2] = 1 << 30
        o = ctx.attention(b.q, b.pool, 1, b.row_offsets, b.kv_len, table)
        assert bool((o[b.offs[2]:b.offs[3]] == 0).all()) and ctx.device_error() == (-5, 2)
    good = Batch(reqs, 4, 2, d, dt, S, seed=4)
    with _ctx(4, 2, d, dt, n=5, pages=good.max_pages) as ctx:
        for kv in (-1, good.max_pages * S + 1):                   # a length out of range: that request is skipped
            out = torch.full_like(good.q, 5.0)
            bad = good.kv_len.clone()
            bad[3] = kv
            ctx.attention(good.q, good.pool, 1, good.row_offsets, bad, good.table, out=out)
            torch.cuda.synchronize()
            assert ctx.device_error() == (-5, 4)
            good.check(out, skip=(3,))
            assert bool((out[good.offs[3]:good.offs[4]] == 5).all())
        out = torch.full_like(good.q, 5.0)                        # more rows than max_new: skipped
        good.run(ctx, 1, out, max_new=50)
        torch.cuda.synchronize()
        assert ctx.device_error() == (-5, 32)
        good.check(out, skip=(1,))
        # row offsets that fall (the last request then owns rows 71 .. 124, the third one's row among them), that
        # pass the end, that are negative
        for offs, skip in (([0, 1, 71, 72, 71, 125], (0, 2, 3, 4)), ([0, 1, 71, 72, 75, 126], (0, 3, 4)),
                           ([-3, 1, 71, 72, 75, 125], (0, 3, 4))):
            out = torch.full_like(good.q, 5.0)
            ctx.attention(good.q, good.pool, 1, _i32(offs), good.kv_len, good.table, out=out)
            torch.cuda.synchronize()
            assert ctx.device_error() == (-5, 32)
            good.check(out, skip=skip)


@pytest.mark.parametrize("dt,d", [(BF, 128), (F32, 64)])
def test_attention_strides_streams_contexts_and_graphs(dt, d):
    reqs = [(1, 70), (90, 260), (2, 2), (33, 33)]
    b = Batch(reqs, 8, 2, d, dt, 16, seed=6, pad=1)
    with _ctx(8, 2, d, dt, n=4, pages=b.max_pages) as ctx, _ctx(8, 2, d, dt, n=9, pages=b.max_pages) as other:
        want = b.run(ctx)
        wide_q = torch.zeros(b.T, 13, d, dtype=dt, device="cuda")
        wide_q[:, 3:11] = b.q
        wide_o = torch.full((b.T, 10, d), 3.0, dtype=dt, device="cuda")
        ctx.attention(wide_q[:, 3:11], b.pool, 1, b.row_offsets, b.kv_len, b.table, out=wide_o[:, 1:9])
        assert torch.equal(wide_o[: b.T - 1, 1:9], want[: b.T - 1])
        assert bool((wide_o[:, [0, 9]] == 3).all()) and bool((wide_o[-1] == 3).all())
        # two contexts at once, each on its own stream
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        outs = [torch.zeros_like(b.q) for _ in range(20)]
        for i, o in enumerate(outs):
            b.run((ctx, other)[i & 1], out=o, stream=(s1, s2)[i & 1])
        torch.cuda.synchronize()
        assert all(torch.equal(o[:-1], want[:-1]) for o in outs)
        # a captured call sees the lengths of each replay
        row_offsets, kv_len, q = b.row_offsets.clone(), b.kv_len.clone(), b.q.clone()
        out = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.attention(q, b.pool, 1, row_offsets, kv_len, b.table, out=out)
        for seed, rq in ((6, reqs), (7, [(1, 1), (100, 200), (0, 0), (20, 31)]), (6, reqs)):
            c = Batch(rq, 8, 2, d, dt, 16, seed=seed, pad=b.T - sum(n for n, _ in rq))
            c.pool, c.table = b.pool, b.table
            if rq is not reqs:  # shorter requests over the same pages
                c.max_pages = b.max_pages
            q.copy_(c.q)
            row_offsets.copy_(c.row_offsets)
            kv_len.copy_(c.kv_len)
            g.replay()
            torch.cuda.synchronize()
            c.check(out)
        assert ctx.device_error() == (0, 0) and other.device_error() == (0, 0)


def test_attention_back_to_back_calls_agree():
    """Hundreds of calls in a row of a batch that uses both kernels, split walks and half-empty tiles: the same
    bits each time and no wait that ran out."""
    rng = random.Random(8)
    reqs = [(rng.choice([1, 1, 1, 40, 70, 200]), 0) for _ in range(24)]
    reqs = [(n, n + rng.randint(0, 900)) for n, _ in reqs]
    b = Batch(reqs, 32, 8, 128, BF, 16, seed=8)
    with _ctx(32, 8, 128, BF, n=24, pages=b.max_pages) as ctx:
        want = b.run(ctx, 32)
        out = torch.zeros_like(want)
        for _ in range(400):
            b.run(ctx, 32, out)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0) and torch.equal(out, want)
        b.check(out, 32)


def test_attention_pool_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are as good as the first."""
    S, hkv, L = 64, 8, 2
    n_pages = (1 << 31) // (L * 2 * hkv * S * 128) + 40
    pool = torch.zeros(n_pages, L, 2, hkv, S, 128, dtype=BF, device="cuda")
    b = Batch([(1, 200), (70, 300)], 16, hkv, 128, BF, S, seed=2)
    last = n_pages - b.pool.shape[0]
    pool[last:] = b.pool
    b.table = torch.where(b.table >= 0, b.table + last, b.table)
    b.pool = pool
    k = torch.randn(3, hkv, 128, device="cuda").to(BF)
    with _ctx(16, hkv, 128, BF, n=2, pages=b.max_pages) as ctx:
        b.check(b.run(ctx))
        slot = _i32([n_pages * S - 1, n_pages * S - 2, 5])
        ctx.qk_norm_rope(torch.zeros(3, 16, 128, dtype=BF, device="cuda"), k, k, pool, 0, _i32([0, 0, 0]), slot)
        torch.cuda.synchronize()
        assert torch.equal(pool[-1, 0, 0, :, -1], k[0]) and torch.equal(pool[-1, 0, 1, :, -2], k[1])
        assert torch.equal(pool[0, 0, 0, :, 5], k[2]) and ctx.device_error() == (0, 0)


# ------------------------------------------------------------------------------------- the run of the three
@pytest.mark.parametrize("dt,d,hq,hkv,mask_block", [(BF, 128, 16, 8, 1), (BF, 128, 8, 2, 32), (F32, 64, 4, 4, 1)])
def test_chunks_then_single_tokens_match_one_pass(dt, d, hq, hkv, mask_block):
    """Prompts in two chunks and then token by token, through plan, cache write and attention, against the same
    rows computed densely in 64 bits from the same projections."""
    S, N, L, mp = 16, 5, 2, 16
    lens = [37, 64, 1, 100, 18]
    splits = [[20, 17], [64, 0], [0, 1], [32, 68], [5, 13]]
    if mask_block > 1:   # a block's keys must be in one chunk: chunks end at block edges
        lens, splits = [32, 64, 32, 96, 64], [[32, 0], [32, 32], [0, 32], [64, 32], [64, 0]]
    singles = 2 if mask_block == 1 else 0
    g = torch.Generator(device="cuda").manual_seed(11)
    total = [n + singles for n in lens]
    proj = [torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").mul_(2).to(dt) for n in total]
    gq, gk = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
    pool = torch.full((48, L, 2, hkv, S, d), float("nan"), dtype=dt, device="cuda")
    free = torch.randperm(48, generator=g, device="cuda").to(torch.int32)
    head, table = _i32([0]), torch.full((N, mp), -1, dtype=torch.int32, device="cuda")
    prefix, got = _i32([0] * N), [torch.zeros(n, hq, d, dtype=dt, device="cuda") for n in total]
    done = [0] * N
    rounds = [[s[i] for s in splits] for i in range(2)] + [[1] * N] * singles
    with _ctx(hq, hkv, d, dt, n=N, pages=mp, layers=L) as ctx:
        T = 260
        plan = ctx.alloc_plan(N, T)
        plan.free_next = head
        for new in rounds:
            ctx.plan(prefix, _i32(new), table, free, head, page_size=S, n_pages=48, out=plan)
            qkv = torch.zeros(T, hq + 2 * hkv, d, dtype=dt, device="cuda")
            at = 0
            for b, n in enumerate(new):
                qkv[at:at + n] = proj[b][done[b]:done[b] + n]
                at += n
            q = ctx.qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pool, 1, plan.row_pos,
                                 plan.row_slot, q_norm=gq, k_norm=gk)
            o = ctx.attention(q, pool, 1, plan.row_offsets, plan.kv_len, table, max_new=max(new), mask_block=mask_block)
            at = 0
            for b, n in enumerate(new):
                got[b][done[b]:done[b] + n] = o[at:at + n]
                at, done[b] = at + n, done[b] + n
            prefix.copy_(plan.kv_len)
        torch.cuda.synchronize()
        assert ctx.device_error() == (0, 0) and done == total
        assert head.item() == sum(_ceil(n, S) for n in total)
    # the dense pass, as a batch whose pool holds the rotated keys rounded to the cache's type
    for b, n in enumerate(total):
        pos = torch.arange(n, device="cuda")
        one = Batch([(n, n)], hq, hkv, d, dt, S, layers=1)
        one.q = _turn64(proj[b][:, :hq], gq, pos, 10000.0, 1e-6)[0].to(dt)
        k = _turn64(proj[b][:, hq:hq + hkv], gk, pos, 10000.0, 1e-6)[0].to(dt)
        pg, at = one.table[0].long()[pos // S], pos % S
        one.pool[pg, 0, 0, :, at], one.pool[pg, 0, 1, :, at] = k, proj[b][:, hq + hkv:]
        # queries and keys were rounded from float32 instead of float64: where that falls on the other side, a stored
        # value moves by one step, 2u, of which few do (float32 work is off by (d + 24) 2^-24, the chance of crossing
        # is that over u); the bound of check() leaves 2u A of a key's weight to spare only in bf16, so the scores
        # get the same allowance through a step of every value
        w_slack = 2 * U[dt]
        ref = torch.zeros_like(one.q)
        with _ctx(hq, hkv, d, dt, n=1, pages=one.max_pages, layers=1) as ctx1:
            ctx1.attention(one.q, one.pool, 0, one.row_offsets, one.kv_len, one.table, mask_block=mask_block, out=ref)
        one.check(ref, mask_block, layer=0)
        q64 = one.q.double()
        B = (q64.abs().sum(-1).amax() * k.double().abs().amax() / math.sqrt(d)).item()
        err = (got[b].double() - ref.double()).abs().max().item()
        crossings = (d + 24) * E / U[dt] if dt == BF else 1.0
        scale = proj[b][:, hq + hkv:].double().abs().max().item()
        assert err <= scale * (2 * U[dt] + 2 * w_slack * B * max(crossings, 2.0 ** -10) + 2.0 ** -7 * (dt == BF)), err
