"""Operators of the prompt-chunk path: what each computes in plain torch, and the calls a user makes.

Three operators put a chunk of new tokens of every request into the paged KV cache and attend over it:

  plan       pages for the new tokens, row offsets, and per token its request, position and cache slot
  qk         per-head RMSNorm of queries and keys (optional), rotate-half RoPE, K and V into the pages
  attention  attention of the new tokens over the paged cache with a block-causal mask

`own` False computes them in elementary torch operations in 32 bits; `own` True calls the library.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases
def _plan(name, requests, new, prefix, rows, page, lens_seed, spare=1.0):
    return dict(name=name, op="plan", requests=requests, new_lo=new[0], new_hi=new[1], prefix_lo=prefix[0],
                prefix_hi=prefix[1], rows=rows, page=page, lens_seed=lens_seed, spare=spare)


def _qk(name, rows, padded, q_heads, kv_heads, dim, dtype, page, norm, lens_seed):
    return dict(name=name, op="qk", rows=rows, padded=padded, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                dtype=dtype, page=page, norm=norm, lens_seed=lens_seed)


def _attn(name, singles, chunks, chunk, ctx, q_heads, kv_heads, dim, dtype, page, mask_block, padded, lens_seed):
    return dict(name=name, op="attention", singles=singles, chunks=chunks, chunk_lo=chunk[0], chunk_hi=chunk[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                mask_block=mask_block, padded=padded, lens_seed=lens_seed)


def listed():
    return [
        # one token for each of 32 running requests: the bookkeeping of every single-token step
        _plan("plan_single_tokens_32", 32, (1, 1), (256, 1024), 32, 64, 11),
        # admission of 256 ragged prompts on top of shared prefixes, more than the pool and the row buffer hold
        _plan("plan_ragged_256", 256, (0, 1024), (0, 2048), 131072, 16, 12, spare=0.9),
        # 32 single tokens of the 16/8-head model: launch latency
        _qk("qk_rows_32", 32, 0, 16, 8, 128, "bf16", 64, True, 21),
        # a full row buffer of the 32/8-head model: 256 requests of 64 tokens
        _qk("qk_rows_16384", 16384, 0, 32, 8, 128, "bf16", 64, True, 22),
        # the model without norms (rotation and cache write alone), a buffer with unused rows at its end
        _qk("qk_rotation_only_4099", 4099, 61, 16, 8, 128, "bf16", 32, False, 23),
        # the float32 model, odd row count, 16-token pages
        _qk("qk_f32_777", 777, 7, 4, 4, 64, "f32", 16, True, 24),
        # single-token attention of 32 requests: a small step, where latency counts
        _attn("attention_single_32", 32, 0, (1, 1), (256, 1024), 16, 8, 128, "bf16", 64, 1, 0, 31),
        # single-token attention of 256 requests, 32/8 heads: the bandwidth-bound serving batch
        _attn("attention_single_256", 256, 0, (1, 1), (512, 2048), 32, 8, 128, "bf16", 64, 1, 0, 32),
        # a fresh prompt of 8192 tokens: compute-bound causal prefill
        _attn("attention_prompt_8192", 0, 1, (8192, 8192), (0, 0), 16, 8, 128, "bf16", 64, 1, 0, 33),
        # running requests and prompt chunks in one batch, block-causal mask, 16-token pages, odd sizes, spare rows
        _attn("attention_mixed_48", 40, 8, (65, 1027), (1, 4096), 32, 8, 128, "bf16", 16, 32, 13, 34),
        # two chunks of a long document over 65 thousand cached tokens
        _attn("attention_long_65536", 0, 2, (1021, 1024), (64000, 65537), 32, 8, 128, "bf16", 64, 1, 0, 35),
        # the float32 model: short prompts and single tokens
        _attn("attention_f32_11", 5, 6, (2, 401), (0, 300), 4, 4, 64, "f32", 16, 1, 3, 36),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: serving batches, prompt chunks and mixtures of both."""
    seed = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64])
    kind = rng.choice(["plan", "qk", "attention", "attention"])
    if kind == "plan":
        n = _log_int(rng, 1, 512)
        hi = rng.choice([1, 64, 512])
        pre = _log_int(rng, 1, 2048)
        rows = max(1, int(n * hi * rng.uniform(0.3, 1.0)))
        case = _plan("", n, (0 if hi > 1 else 1, hi), (0, pre), min(rows, 131072), page, seed,
                     rng.choice([1.0, 1.0, 0.7]))
    elif kind == "qk":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        hq, hkv = rng.choice([(16, 8), (32, 8), (4, 4), (6, 2), (8, 1)])
        dim = 128 if dtype == "bf16" else rng.choice([64, 128])
        rows = _log_int(rng, 1, 12000 if dtype == "bf16" else 3000)
        case = _qk("", rows, rng.choice([0, 0, 1, 17]), hq, hkv, dim, dtype, page, rng.random() < 0.7, seed)
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        hq, hkv = rng.choice([(16, 8), (32, 8), (4, 4), (6, 2), (8, 1)])
        dim = 128 if dtype == "bf16" else rng.choice([64, 128])
        mask_block = rng.choice([1, 1, 16, 32, 64, 100])
        mix = rng.choice(["single", "chunk", "mixed"])
        top = 8192 if dtype == "bf16" else 1500
        if mix == "single":
            n = _log_int(rng, 1, 200)
            ctx = _log_int(rng, 1, min(65536, 300000 // n) if dtype == "bf16" else 2000)
            case = _attn("", n, 0, (1, 1), (ctx // 3, ctx), hq, hkv, dim, dtype, page, mask_block, 0, seed)
        elif mix == "chunk":
            n = rng.randint(1, 3)
            new = _log_int(rng, 2, top // (2 * n))
            ctx = _log_int(rng, 1, top)
            case = _attn("", 0, n, (max(2, new // 2), new), (0, ctx), hq, hkv, dim, dtype, page, mask_block,
                         rng.choice([0, 5]), seed)
        else:
            n = _log_int(rng, 2, 40)
            new = _log_int(rng, 2, top // 16)
            ctx = _log_int(rng, 1, top // 4)
            case = _attn("", n, rng.randint(1, 6), (2, new + 1), (0, ctx), hq, hkv, dim, dtype, page, mask_block,
                         rng.choice([0, 9]), seed)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------- lengths
def _plan_lens(case):
    rng = random.Random(case["lens_seed"])
    prefix = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["requests"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    return prefix, new


def _attn_lens(case):
    """(new tokens, cached tokens before them) of each request, single tokens and chunks interleaved."""
    rng = random.Random(case["lens_seed"])
    reqs = [(1, rng.randint(case["ctx_lo"], case["ctx_hi"])) for _ in range(case["singles"])]
    reqs += [(rng.randint(case["chunk_lo"], case["chunk_hi"]), rng.randint(case["ctx_lo"], case["ctx_hi"]))
             for _ in range(case["chunks"])]
    rng.shuffle(reqs)
    return reqs


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "qk": _prepare_qk, "attention": _prepare_attn}[case["op"]](case, gen)


def _context(case, requests, max_pages):
    """The handle a user's program keeps (only when the library's calls are timed)."""
    if not own:
        return None
    from decodability_aware_token_b200 import ChunkContext
    return ChunkContext(n_layers=2, n_q_heads=case.get("q_heads", 16), n_kv_heads=case.get("kv_heads", 8),
                        head_dim=case.get("dim", 128), dtype=_DTYPES[case.get("dtype", "bf16")],
                        max_requests=requests, max_pages_per_req=max_pages, rope_theta=10000.0, device="cuda:0")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_plan(case, gen):
    prefix, new = _plan_lens(case)
    S, N = case["page"], case["requests"]
    have = [_ceil(p, S) for p in prefix]
    total = sum(have)
    wanted = sum(_ceil(p + n, S) for p, n in zip(prefix, new)) - total
    n_free = int(wanted * case["spare"]) + 2
    n_pages = total + n_free
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    max_pages = _ceil(max(p + n for p, n in zip(prefix, new)), S) + 1
    have_t = torch.tensor(have, device="cuda")
    cols = torch.arange(max_pages, device="cuda")[None]
    base = torch.cumsum(have_t, 0) - have_t
    idx = (base[:, None] + cols).clamp(max=n_pages - 1)
    table = torch.where(cols < have_t[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous()
    ctx = _context(case, N, max_pages)
    return dict(case=case, prefix_len=_i32(prefix), new_len=_i32(new), page_table=table,
                free_pages=order[total:].clone(), free_head=_i32([1]), n_pages=n_pages, ctx=ctx,
                plan=ctx.alloc_plan(N, case["rows"]) if ctx else None)


def _prepare_qk(case, gen):
    T, hq, hkv, d, S = case["rows"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    dt = _DTYPES[case["dtype"]]
    live = T - min(case["padded"], T - 1)
    n_pages = _ceil(live, S) + 2
    # what the QKV projection leaves: one row per token, query heads, key heads, value heads
    qkv = torch.randn(T, hq + 2 * hkv, d, generator=gen, device="cuda", dtype=torch.float32).mul_(1.5).to(dt)
    rng = random.Random(case["lens_seed"])
    start = rng.randint(0, 2000) if live < 4000 else rng.randint(0, 100000)
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[:live] = torch.arange(live, device="cuda", dtype=torch.int32) + start
    slot = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    # consecutive tokens fill pages in a scattered page order
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(live, device="cuda")
    slot[:live] = order[at // S] * S + (at % S).to(torch.int32)
    pool = torch.randn(n_pages, 2, 2, hkv, S, d, generator=gen, device="cuda", dtype=torch.float32).to(dt)
    gain = [(1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt) if case["norm"] else None for _ in range(2)]
    return dict(case=case, qkv=qkv, row_pos=pos, row_slot=slot, kv_pool=pool, q_norm=gain[0], k_norm=gain[1],
                out=torch.zeros(T, hq, d, dtype=dt, device="cuda"), ctx=_context(case, 1, 1))


def _prepare_attn(case, gen):
    reqs = _attn_lens(case)
    hq, hkv, d, S = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    dt = _DTYPES[case["dtype"]]
    new = [r[0] for r in reqs]
    kv_len = [r[0] + r[1] for r in reqs]
    need = [_ceil(k, S) for k in kv_len]
    n_pages = sum(need) + 3
    max_pages = max(need) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(reqs), max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    T = offs[-1] + case["padded"]
    pool = torch.randn(n_pages, 2, 2, hkv, S, d, generator=gen, device="cuda", dtype=dt)
    # normed and rotated queries; a gain above 1, so that attention picks some keys out
    q = torch.randn(T, hq, d, generator=gen, device="cuda", dtype=torch.float32).mul_(2.0).to(dt)
    return dict(case=case, q=q, kv_pool=pool, layer=1, row_offsets=_i32(offs), kv_len=_i32(kv_len), page_table=table,
                max_new=max(new), out=torch.zeros(T, hq, d, dtype=dt, device="cuda"), new_host=new, kv_host=kv_len,
                ctx=_context(case, len(reqs), max_pages))


# ----------------------------------------------------------------------------------------------- runs
def run(state):
    return {"plan": _run_plan, "qk": _run_qk, "attention": _run_attn}[state["case"]["op"]](state)


def _run_plan(s):
    S, T = s["case"]["page"], s["case"]["rows"]
    if own:
        p = s["ctx"].plan(s["prefix_len"], s["new_len"], s["page_table"], s["free_pages"], s["free_head"],
                          page_size=S, n_pages=s["n_pages"], out=s["plan"])
        return [p.row_offsets, p.kv_len, p.row_req, p.row_pos, p.row_slot, s["page_table"], p.free_next]
    prefix, new, table = s["prefix_len"].long(), s["new_len"].long(), s["page_table"]
    free, head = s["free_pages"], s["free_head"].long()
    have = (prefix + S - 1) // S
    rows_ok = (new == 0) | (torch.cumsum(new, 0) <= T)
    need = ((prefix + new + S - 1) // S - have) * rows_ok
    cum = torch.cumsum(need, 0)
    placed = rows_ok & ((need == 0) | (cum <= free.shape[0] - head))
    taken, rows = need * placed, new * placed
    offs = torch.cat([torch.zeros_like(head), torch.cumsum(rows, 0)])
    cols = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (cols >= have[:, None]) & (cols < (have + taken)[:, None])
    src = (head + (cum - need)[:, None] + cols - have[:, None]).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(fresh, free[src], table))
    r = torch.arange(T, device=table.device)
    b = torch.searchsorted(offs, r, right=True) - 1
    live = r < offs[-1]
    b = b.clamp(max=new.shape[0] - 1)
    pos = prefix[b] + r - offs[b]
    page = table[b, (pos // S).clamp(max=table.shape[1] - 1)].long()
    slot = torch.where((page >= 0) & (page < s["n_pages"]), page * S + pos % S, torch.full_like(page, -1))
    pad = torch.full_like(r, -1)
    out = [offs, prefix + rows, torch.where(live, b, pad), torch.where(live, pos, pad), torch.where(live, slot, pad)]
    return [x.to(torch.int32) for x in out] + [table, (head + taken.sum()).to(torch.int32)]


def _run_qk(s):
    c = s["case"]
    hq, hkv, d, S = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    qkv, pool, layer = s["qkv"], s["kv_pool"], 1
    if own:
        s["ctx"].qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pool, layer, s["row_pos"],
                              s["row_slot"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, out=s["out"])
        return [s["out"], pool]
    live = s["row_pos"] >= 0
    pos = s["row_pos"].clamp(min=0)
    inv = 10000.0 ** (-torch.arange(0, d, 2, device=qkv.device, dtype=torch.float64) / d)
    ang = pos.double()[:, None] * inv
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turn(x, gain):
        x = x.float()
        if gain is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.float()
        lo, hi = x[..., : d // 2], x[..., d // 2:]
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)

    q = turn(qkv[:, :hq], s["q_norm"]).to(qkv.dtype)
    k = turn(qkv[:, hq:hq + hkv], s["k_norm"]).to(qkv.dtype)
    s["out"].copy_(torch.where(live[:, None, None], q, s["out"]))
    keep = torch.nonzero(s["row_slot"] >= 0)[:, 0]
    slot = s["row_slot"][keep].long()
    pool[slot // S, layer, 0, :, slot % S] = k[keep]
    pool[slot // S, layer, 1, :, slot % S] = qkv[keep, hq + hkv:]
    return [s["out"], pool]


def _run_attn(s):
    c = s["case"]
    hq, hkv, d, S, mb = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["mask_block"]
    q, pool, layer, out = s["q"], s["kv_pool"], s["layer"], s["out"]
    if own:
        s["ctx"].attention(q, pool, layer, s["row_offsets"], s["kv_len"], s["page_table"], max_new=s["max_new"],
                           mask_block=mb, out=out)
        return out
    G, row = hq // hkv, 0
    for b, (n, kv) in enumerate(zip(s["new_host"], s["kv_host"])):
        pages = s["page_table"][b, : _ceil(kv, S)].long()
        pos = torch.arange(kv - n, kv, device=q.device)
        seen = torch.arange(kv, device=q.device)[None] < ((pos // mb + 1) * mb)[:, None]     # [n, kv]
        group = hkv if n * kv * hq < (1 << 28) else 1
        for g in range(0, hkv, group):
            kk = pool[pages, layer, 0, g:g + group].transpose(0, 1).reshape(group, -1, d)[:, :kv].float()
            vv = pool[pages, layer, 1, g:g + group].transpose(0, 1).reshape(group, -1, d)[:, :kv].float()
            qq = q[row:row + n, g * G:(g + group) * G].float().reshape(n, group, G, d).permute(1, 2, 0, 3)
            sc = torch.matmul(qq, kk[:, None].transpose(-1, -2)) / math.sqrt(d)              # [group, G, n, kv]
            sc = sc.masked_fill_(~seen, float("-inf"))
            sc = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(sc, vv[:, None]) / sc.sum(-1, keepdim=True)
            out[row:row + n, g * G:(g + group) * G] = o.permute(2, 0, 1, 3).reshape(n, group * G, d).to(out.dtype)
        row += n
    return out


# ----------------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        prefix, new = _plan_lens(case)
        S = case["page"]
        pages = sum(_ceil(p + n, S) - p // S for p, n in zip(prefix, new))  # entries read or written
        return {"bytes": 4 * (3 * case["rows"] + 4 * case["requests"] + 2 * pages), "flops": 8 * case["rows"]}
    if case["op"] == "qk":
        e = 2 if case["dtype"] == "bf16" else 4
        live = case["rows"] - min(case["padded"], case["rows"] - 1)
        vec = (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": live * (2 * vec * e + 8), "flops": live * vec * 8}
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d, mb = case["q_heads"], case["kv_heads"], case["dim"], case["mask_block"]
    rows = keys = seen = 0
    for n, ctx in _attn_lens(case):
        rows += n
        keys += n + ctx
        seen += sum(min(n + ctx, ((ctx + i) // mb + 1) * mb) for i in range(n))
    return {"bytes": e * (keys * hkv * d * 2 + rows * hq * d * 2), "flops": 4 * hq * d * seen}


# ---------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"plan": _exact_plan, "qk": _exact_qk, "attention": _exact_attn}[case["op"]](case, s)


def _exact_plan(case, s):
    """Request by request on the host."""
    S, T = case["page"], case["rows"]
    prefix, new = s["prefix_len"].tolist(), s["new_len"].tolist()
    table, free, head = s["page_table"].tolist(), s["free_pages"].tolist(), s["free_head"].tolist()[0]
    offs, kv, req, pos, slot = [0], [], [], [], []
    asked_rows, asked_pages, at = 0, 0, head
    for b, (p, n) in enumerate(zip(prefix, new)):
        asked_rows += n
        fits = n == 0 or asked_rows <= T
        have = _ceil(p, S)
        need = _ceil(p + n, S) - have if fits else 0
        asked_pages += need
        if need > 0 and asked_pages > len(free) - head:
            fits = False
        if not fits:
            n = need = 0
        for i in range(need):
            table[b][have + i] = free[at]
            at += 1
        for i in range(n):
            page = table[b][(p + i) // S]
            req.append(b)
            pos.append(p + i)
            slot.append(page * S + (p + i) % S if 0 <= page < s["n_pages"] else -1)
        offs.append(len(req))
        kv.append(p + n)
    pad = [-1] * (T - len(req))
    return [_i32(offs), _i32(kv), _i32(req + pad), _i32(pos + pad), _i32(slot + pad), _i32(table), _i32([at])]


def _exact_qk(case, s):
    """Pairs (i, i + d/2) as complex numbers turned by exp(i pos theta^(-2i/d)), in float64."""
    hq, hkv, d, S = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    live = torch.nonzero(s["row_pos"] >= 0).flatten()
    x = s["qkv"][live].double()
    freq = torch.exp(torch.arange(d // 2, device=x.device, dtype=torch.float64) * (-2.0 * math.log(10000.0) / d))
    ang = torch.outer(s["row_pos"][live].double(), freq)
    unit = torch.polar(torch.ones_like(ang), ang)[:, None]

    def turned(v, gain):
        if gain is not None:
            v = v / torch.sqrt(v.square().sum(-1, keepdim=True) / d + 1e-6) * gain.double()
        z = torch.complex(v[..., : d // 2].contiguous(), v[..., d // 2:].contiguous()) * unit
        return torch.cat([z.real, z.imag], dim=-1)

    out = s["out"].double()
    out[live] = turned(x[:, :hq], s["q_norm"])
    pool = s["kv_pool"].double()
    slot = s["row_slot"][live].long()
    stored = slot >= 0
    page, off = slot[stored] // S, slot[stored] % S
    pool[page, 1, 0, :, off] = turned(x[:, hq:hq + hkv], s["k_norm"])[stored]
    pool[page, 1, 1, :, off] = x[stored][:, hq + hkv:]
    return [out, pool]


def _exact_attn(case, s):
    """Head by head, rows in slices, in float64."""
    hq, hkv, d, S, mb = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["mask_block"]
    G, row = hq // hkv, 0
    out = s["out"].double()
    for b, (n, kv) in enumerate(zip(s["new_host"], s["kv_host"])):
        pages = s["page_table"][b, : _ceil(kv, S)].long()
        j = torch.arange(kv, device=out.device)
        for h in range(hkv):
            keys = s["kv_pool"][pages, 1, 0, h].reshape(-1, d)[:kv].double()
            vals = s["kv_pool"][pages, 1, 1, h].reshape(-1, d)[:kv].double()
            step = max(1, (1 << 27) // (kv * G))
            for r0 in range(0, n, step):
                r1 = min(n, r0 + step)
                qs = s["q"][row + r0:row + r1, h * G:(h + 1) * G].double().reshape(-1, d)
                first_hidden = ((torch.arange(kv - n + r0, kv - n + r1, device=out.device) // mb + 1) * mb)
                hidden = j[None] >= first_hidden.repeat_interleave(G)[:, None]
                logits = (qs @ keys.T).div_(d ** 0.5).masked_fill_(hidden, -torch.inf)
                w = torch.softmax(logits, dim=-1)
                out[row + r0:row + r1, h * G:(h + 1) * G] = (w @ vals).reshape(-1, G, d)
        row += n
    return out
