"""The chunk operators' two host paths (csrc/marshal.cpp and chunk.py): what one takes the other takes, with the same
results, and a refused call is refused in the same words."""
import pytest
import torch

from decodability_aware_token_b200 import ChunkContext, _abi

HQ, HKV, D, L, S, PAGES, MP, N, ROWS = 4, 2, 128, 2, 16, 12, 4, 3, 40
BF = torch.bfloat16


def test_anything_but_cuda_tensors_is_left_to_the_python_path():
    m, entry = _abi.load_marshal()
    assert m.torch_version == torch.__version__.split("+")[0]
    t = torch.zeros(2, dtype=torch.int32)
    assert m.plan(1, 2) is None and m.qk() is None and m.attention(None) is None
    for bad in (t, t.double(), None, "x", 3, torch.zeros(2, dtype=torch.int32, device="meta"), t.to_sparse()):
        # (no entry point is called: the tensors are refused first)
        assert m.plan(entry[0], 0, 0, 0, MP, S, PAGES, *[bad] * 11) is None
        assert m.qk(entry[1], 0, 0, 0, True, HQ, HKV, D, L, 0, 1e-6, *[bad] * 9) is None
        assert m.attention(entry[2], 0, 0, 0, True, HQ, HKV, D, L, MP, 0, 1, 1, 0.0, *[bad] * 6) is None
    for page_size in (1 << 40, -(1 << 40), 1 << 70, 1.5, "x", None):
        assert m.plan(entry[0], 0, 0, 0, MP, page_size, PAGES, *[t] * 11) is None


def _state(dev):
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(BF).to(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    st = dict(prefix_len=i32([0, 17, 5]), new_len=i32([20, 1, 9]), free_pages=i32(list(range(3, PAGES))), free_head=i32([0]),
              page_table=i32([[-1] * MP, [0, 1, -1, -1], [2, -1, -1, -1]]), q=rnd(ROWS, HQ, D), k=rnd(ROWS, HKV, D),
              v=rnd(ROWS, HKV, D), kv_pool=rnd(PAGES, L, 2, HKV, S, D), q_norm=rnd(D), k_norm=rnd(D),
              out=rnd(ROWS, HQ, D), o=rnd(ROWS, HQ, D))
    return st


def _ctx():
    return ChunkContext(n_layers=L, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D, max_requests=N, max_pages_per_req=MP)


def _plan(ctx, st, out, **kw):
    return ctx.plan(*(st[k] for k in ("prefix_len", "new_len", "page_table", "free_pages", "free_head")), page_size=S,
                    n_pages=PAGES, out=out, **kw)


def _run(ctx, st, plan, **kw):
    _plan(ctx, st, plan, **kw)
    ctx.qk_norm_rope(st["q"], st["k"], st["v"], st["kv_pool"], 1, plan.row_pos, plan.row_slot, q_norm=st["q_norm"],
                     k_norm=st["k_norm"], out=st["out"], **kw)
    ctx.attention(st["out"], st["kv_pool"], 1, plan.row_offsets, plan.kv_len, st["page_table"], max_new=ROWS, out=st["o"], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("side", [False, True])
def test_both_paths_give_the_same_results(side):
    with _ctx() as ctx:
        native, res = ctx._marshal, []
        stream = torch.cuda.Stream() if side else None
        for m in (native, None):
            st, plan = _state("cuda"), ctx.alloc_plan(N, ROWS)
            ctx._marshal = m
            torch.cuda.synchronize()
            _run(ctx, st, plan, **(dict(stream=stream) if side else {}))
            torch.cuda.synchronize()
            assert ctx.device_error() == (0, 0)
            res.append([plan.row_offsets, plan.kv_len, plan.row_req, plan.row_pos, plan.row_slot, plan.free_next,
                        st["page_table"], st["out"], st["kv_pool"], st["o"]])
        assert all(torch.equal(a, b) for a, b in zip(*res))
        assert res[0][0].tolist() == [0, 20, 21, 30]


def _bad_cases():
    odd = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)              # off by one element
    wide = lambda t: torch.cat([t, t], -1)[..., : t.shape[-1]]                                # heads not dense
    skew = lambda t: torch.zeros(t.numel() + 4 * len(t), dtype=t.dtype, device=t.device).as_strided(
        t.shape, (t.stride(0) + 4, t.stride(1), 1))                                           # rows not aligned
    overlap = lambda t: t.as_strided(t.shape, (t.stride(0) - 8, t.stride(1), 1))
    for name in ("prefix_len", "new_len", "page_table", "free_pages", "free_head"):
        yield "plan", name, "long", lambda t: t.long()
        yield "plan", name, "host", lambda t: t.cpu()
        yield "plan", name, "strided", lambda t: torch.stack([t, t], -1)[..., 0]
    yield "plan", "new_len", "short", lambda t: t[:-1]
    yield "plan", "free_head", "two", lambda t: torch.cat([t, t])
    yield "plan", "page_table", "list", lambda t: t.tolist()
    for name in ("q", "k", "v", "out"):
        for what, f in (("float", lambda t: t.float()), ("host", lambda t: t.cpu()), ("odd", odd), ("wide", wide), ("skew", skew),
                        ("overlap", overlap), ("flat", lambda t: t.flatten(1)), ("none", lambda t: None)):
            if what == "none" and name in ("q", "out"):
                continue  # (None for out is allocated; q gives the number of rows)
            yield "qk", name, what, f
    for name in ("q_norm", "k_norm"):
        for what, f in (("float", lambda t: t.float()), ("odd", odd), ("short", lambda t: t[:-1])):
            yield "qk", name, what, f
    for op in ("qk", "attention"):
        for what, f in (("float", lambda t: t.float()), ("odd", odd), ("layers", lambda t: t[:, :1]),
                        ("swapped", lambda t: t.transpose(3, 4)), ("5d", lambda t: t[0])):
            yield op, "kv_pool", what, f
    yield "attention", "q", "odd", odd
    yield "attention", "o", "wide", wide
    yield "attention", "page_table", "wide", lambda t: torch.cat([t, t], 1)


@pytest.mark.gpu
@pytest.mark.parametrize("op,name,what,change", [pytest.param(*c, id="-".join(c[:3])) for c in _bad_cases()])
def test_both_paths_refuse_in_the_same_words(op, name, what, change):
    with _ctx() as ctx:
        native, said = ctx._marshal, []
        for m in (native, None):
            st, plan = _state("cuda"), ctx.alloc_plan(N, ROWS)
            _plan(ctx, st, plan)
            st[name] = change(st[name])
            ctx._marshal = m
            if (name, what) == ("free_head", "strided"):
                assert st[name].is_contiguous()  # one element: its stride means nothing, and both paths take it
                _plan(ctx, st, plan)
                continue
            with pytest.raises((TypeError, ValueError)) as e:
                if op == "plan":
                    _plan(ctx, st, plan)
                elif op == "qk":
                    ctx.qk_norm_rope(st["q"], st["k"], st["v"], st["kv_pool"], 1, plan.row_pos, plan.row_slot,
                                     q_norm=st["q_norm"], k_norm=st["k_norm"], out=st["out"])
                else:
                    ctx.attention(st["q"], st["kv_pool"], 1, plan.row_offsets, plan.kv_len, st["page_table"],
                                  max_new=ROWS, out=st["o"])
            said.append((e.type, str(e.value)))
        assert said[:1] == said[1:]


@pytest.mark.gpu
def test_both_paths_refuse_numbers_alike():
    calls = [lambda c, s, p: c.qk_norm_rope(s["q"], s["k"], s["v"], s["kv_pool"], L, p.row_pos, p.row_slot, out=s["out"]),
             lambda c, s, p: c.qk_norm_rope(s["q"], s["k"], s["v"], s["kv_pool"], -1, p.row_pos, p.row_slot, out=s["out"]),
             lambda c, s, p: c.qk_norm_rope(s["q"], s["k"], s["v"], s["kv_pool"], 0, p.row_pos, p.row_slot, eps=-1.0, out=s["out"]),
             lambda c, s, p: c.attention(s["q"], s["kv_pool"], 0, p.row_offsets, p.kv_len, s["page_table"], max_new=0, out=s["o"]),
             lambda c, s, p: c.attention(s["q"], s["kv_pool"], 0, p.row_offsets, p.kv_len, s["page_table"], max_new=4,
                                         mask_block=0, out=s["o"]),
             lambda c, s, p: c.attention(s["q"], s["kv_pool"], 0, p.row_offsets, p.kv_len, s["page_table"], max_new=4,
                                         scale=-1.0, out=s["o"]),
             lambda c, s, p: c.attention(s["q"], s["kv_pool"], 0, p.row_offsets, p.kv_len, s["page_table"], max_new=4, out=s["q"]),
             lambda c, s, p: c.plan(s["prefix_len"], s["new_len"], s["page_table"], s["free_pages"], s["free_head"],
                                    page_size=0, n_pages=PAGES, out=p),
             lambda c, s, p: c.plan(s["prefix_len"], s["new_len"], s["page_table"], s["free_pages"], s["free_head"],
                                    page_size=1 << 33, n_pages=PAGES, out=p)]
    with _ctx() as ctx:
        native, st, plan = ctx._marshal, _state("cuda"), ctx.alloc_plan(N, ROWS)
        for call in calls:
            said = []
            for m in (native, None):
                ctx._marshal = m
                with pytest.raises(Exception) as e:
                    call(ctx, st, plan)
                said.append((e.type, str(e.value)))
            assert said[0] == said[1]
        ctx._marshal = native
        ctx.close()
        with pytest.raises(ValueError, match="closed"):
            _plan(ctx, st, plan)
