"""cvr_kv_tables and cvr_kv_append against their definitions: exact integers and exact rows; then decode steps of tables,
append and attend together, as a serving loop runs them, and the cache against the scoring path's own cross-attention."""
import math
import random

import pytest

from kv_util import Cache, assert_within, cvr_type, pool, tables_reference, torch_type

pytestmark = pytest.mark.gpu


def dev(x, kind="int32"):
    import torch
    return torch.tensor(x, dtype=getattr(torch, kind), device="cuda")


def run_tables(lens, new, held, free, head, table, page, n_slots, n_pages, max_pages, give_all=True):
    import torch
    import cvr_ranking_model_gb300 as cvr
    n = len(lens)
    kv = cvr.KvCache(cvr.make_kv_config(1, 1, 32, page, n_pages, max(n, 1), max_pages))
    t = dev(table).reshape(-1, max_pages)
    t_all = torch.cat([t, torch.full((1, max_pages), 77, dtype=torch.int32, device="cuda")])
    pages, head_out = dev([-5] * (n + 1)), dev([-5, -5])
    slots = dev([-9] * (n_slots + 1), "int64")
    a = [dev(x if x is not None else [0]) for x in (lens, new, held, free or [0], [head])]
    kv.tables(n, a[0].data_ptr(), t_all.data_ptr(), new_lens=a[1].data_ptr() if new is not None else 0,
              held=a[2].data_ptr() if held is not None else 0, free_pages=a[3].data_ptr(), n_free=len(free),
              free_head=a[4].data_ptr() if give_all else 0, pages=pages.data_ptr() if give_all else 0,
              free_head_out=head_out.data_ptr() if give_all else 0, slots=slots.data_ptr() if n_slots else 0, n_slots=n_slots)
    st = kv.sync(check=False)
    for x, y in zip(a, (lens, new, held, free or [0], [head])):
        assert y is None or x.tolist() == list(y)  # a call leaves its inputs as they were
    assert t_all[-1].tolist() == [77] * max_pages and int(slots[-1]) == -9 and int(pages[-1]) == -5 and int(head_out[1]) == -5
    return t_all[:-1].tolist(), pages[:-1].tolist(), int(head_out[0]), slots[:-1].tolist(), st


@pytest.mark.parametrize("n,max_len,page", [(1, 1, 8), (1, 5000, 16), (3, 40, 8), (64, 300, 16), (700, 90, 32), (1023, 20, 8), (1024, 20, 8),
                                            (1025, 20, 8), (5000, 17, 256), (2500, 400, 64), (511, 700, 8), (512, 9, 8), (513, 9, 8),
                                            (20000, 30, 8), (2, 150000, 32)])
@pytest.mark.parametrize("step", ["decode", "fill", "mixed"])
def test_tables(n, max_len, page, step):
    rng = random.Random(n * 1000 + page)
    max_pages = -(-max_len // page) + 1
    lens = [rng.choice([0, 1, rng.randint(0, max_len), max_len]) for _ in range(n)]
    new = [x if step == "fill" else min(x, 1) if step == "decode" else rng.randint(0, x) for x in lens]
    held = [-(-(x - y) // page) for x, y in zip(lens, new)]
    if step == "mixed":  # pages held ahead of need stay
        held = [min(max_pages, h + rng.choice([0, 0, 1])) for h in held]
    n_pages = sum(held) + sum(-(-x // page) for x in lens) + 10
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [rng.randint(-99, -1) for _ in range(max_pages - h)])
        at += h
    free, head = ids[:2] + ids[at:], 2
    n_slots = sum(new) + rng.choice([0, 1, 300])
    want = tables_reference(lens, new, held, free, head, table, page, n_slots)
    got = run_tables(lens, new, held, free, head, table, page, n_slots, n_pages, max_pages)
    assert got[4] == 0
    for g, w, what in zip(got, want, ("table", "pages", "head", "slots")):
        assert g == w, what


def test_tables_defaults_and_nothing_to_do():
    got = run_tables([5, 0, 20], None, None, [4, 3, 2, 1], 0, [[9, 9, 9]] * 3, 16, 3, 10, 3, give_all=False)
    assert got[0] == [[4, 9, 9], [9, 9, 9], [3, 2, 9]] and got[3] == [4 * 16 + 4, 2 * 16 + 3, -1] and got[4] == 0
    got = run_tables([5], [5], [1], [], 0, [[7, 9, 9]], 16, 0, 10, 3)
    assert got[0] == [[7, 9, 9]] and got[1] == [1] and got[4] == 0
    import cvr_ranking_model_gb300 as cvr
    kv = cvr.KvCache(cvr.make_kv_config(1, 1, 32, 16, 10, 4, 4))
    head, slots = dev([3, 0]), dev([0, 0], "int64")
    kv.tables(0, 0, 0, free_pages=dev([1] * 9).data_ptr(), n_free=9, free_head=head.data_ptr(), free_head_out=head.data_ptr() + 4,
              slots=slots.data_ptr(), n_slots=2)
    kv.sync()
    assert head.tolist() == [3, 3] and slots.tolist() == [-1, -1]


def test_tables_when_the_free_list_ends():
    lens, free = [20, 5, 40], [3, 1, 2]
    want = tables_reference(lens, lens, [0] * 3, free, 0, [[9] * 4] * 3, 16, 70)
    got = run_tables(lens, lens, [0] * 3, free, 0, [[9] * 4] * 3, 16, 70, 10, 4)
    assert got[4] == 8 and got[:4] == want
    assert want[1] == [2, 1, 0] and want[0][2] == [-1, -1, -1, 9]


@pytest.mark.parametrize("page,left", [(8, 0), (8, 1), (8, 700), (8, 1250), (64, 90), (256, 21)])
def test_long_histories_when_the_free_list_ends(page, left):
    lens, held_tokens = [6000, 0, 1, 5003, 300], [100, 0, 0, 3, 300]
    held = [-(-x // page) for x in held_tokens]
    new = [x - y for x, y in zip(lens, held_tokens)]
    max_pages = -(-6000 // page) + 2
    ids = list(range(2000))
    random.Random(page + left).shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (max_pages - h))
        at += h
    free = ids[at:at + left]
    want = tables_reference(lens, new, held, free, 0, table, page, sum(new) + 5)
    got = run_tables(lens, new, held, free, 0, table, page, sum(new) + 5, 2000, max_pages)
    assert got[4] == (8 if left < sum(max(0, -(-x // page) - h) for x, h in zip(lens, held)) else 0)
    for g, w, what in zip(got, want, ("table", "pages", "head", "slots")):
        assert g == w, what


def test_tables_report_bad_inputs():
    base = dict(lens=[20, 5], new=[1, 1], held=[1, 0], free=[3, 1, 2], head=0, table=[[5, 9], [9, 9]], page=16, n_slots=4, n_pages=10, max_pages=2)
    assert run_tables(**base)[4] == 0
    for st, change in ((6, dict(lens=[33, 5])), (6, dict(lens=[-1, 5])), (6, dict(new=[21, 1])), (6, dict(new=[-1, 1])), (6, dict(held=[3, 0])),
                       (6, dict(held=[-1, 0])), (6, dict(head=4)), (6, dict(head=-1)), (6, dict(n_slots=1)), (3, dict(free=[10, 1, 2])),
                       (3, dict(free=[-2, 1, 2])), (3, dict(table=[[10, 9], [9, 9]], lens=[16, 5])), (8, dict(free=[3]))):
        assert run_tables(**{**base, **change})[4] == st, change
    got = run_tables(**{**base, "n_slots": 1})
    assert got[3] == [3 * 16 + 3]
    # the list's second entry was asked for, and only the first request's page was bad
    got = run_tables(**{**base, "free": [10, 1, 2]})
    assert got[0] == [[5, -1], [1, 9]] and got[3] == [-1, 1 * 16 + 4, -1, -1]


def test_tables_refusals():
    import cvr_ranking_model_gb300 as cvr
    kv = cvr.KvCache(cvr.make_kv_config(1, 1, 32, 16, 10, 4, 4))
    x = dev([0] * 64)
    p = x.data_ptr()
    ok = dict(n_req=2, lens=p, table=p + 64)
    for st, change in ((2, dict(n_req=5)), (2, dict(n_req=-1)), (1, dict(lens=0)), (1, dict(table=0)), (1, dict(n_free=1)), (2, dict(n_free=-1)),
                       (1, dict(n_slots=1)), (2, dict(n_slots=-1)), (1, dict(held=p, pages=p)), (1, dict(free_head=p, free_head_out=p))):
        with pytest.raises(cvr.CvrError) as e:
            kv.tables(**{**ok, **change})
        assert e.value.status == st, change


# ---- append ----
def quantised(x):
    """(codes, scales) of rows [..., dim] by the definition, in 64 bits."""
    import torch
    big = x.double().abs().amax(-1, keepdim=True)
    return torch.round(x.double() * 127 / torch.where(big == 0, 1.0, big)), big[..., 0] / 127


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "i8"), ("f16", "i8")])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("layout,heads,n,page,shared", [("page", 1, 1, 8, False), ("token", 3, 100, 16, False), ("gaps", 8, 777, 32, False),
                                                        ("page", 5, 64, 256, True), ("token", 2, 5000, 64, False)])
def test_append(dtype, cache, dim, layout, heads, n, page, shared):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + dim)
    kind = "i8" if cache == "i8" else dtype
    n_pages = -(-n // page) + 3
    names = ["k"] if shared else ["k", "v"]
    pools = {x: pool(n_pages, heads, page, dim, kind, layout) for x in names}
    for x in names:
        (pools[x] if pools[x]._base is None else pools[x]._base).zero_()  # the values between rows too
    scales = {x: torch.full((n_pages, heads, page), 5.0, device="cuda") for x in names} if kind == "i8" else {}
    import cvr_ranking_model_gb300 as cvr
    args = dict(k=pools["k"].data_ptr(), k_strides=pools["k"].stride()[:3])
    if scales:
        args["k_scale"] = scales["k"].data_ptr()
    if not shared:
        args.update(v=pools["v"].data_ptr(), v_strides=pools["v"].stride()[:3], v_scale=scales["v"].data_ptr() if scales else 0)
    kv = cvr.KvCache(cvr.make_kv_config(heads, heads, dim, page, n_pages, 1, 1, cvr_type(dtype), cvr_type(kind), **args))
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:n]
    slots[torch.rand(n, generator=gen, device="cuda") < 0.1] = -1  # padding
    wide = torch.randn((n, 2 * heads * dim + 24), generator=gen, device="cuda").to(torch_type(dtype))
    if n > 3:  # a zero row, one whose values lie far apart and halves of steps
        wide[0] = 0
        wide[1, ::2] *= 1e-3 if dtype == "f16" else 1e-20
        wide[2] = torch.arange(wide.shape[1], device="cuda").remainder(255).sub(127).to(wide.dtype) / 2
    rows = {"k": wide[:, 8:8 + heads * dim], "v": wide[:, 16 + heads * dim:16 + 2 * heads * dim]}
    want = {x: pools[x].clone() for x in names}
    want_s = {x: scales[x].clone() for x in scales}
    on = slots >= 0
    for x in names:
        val = rows[x].reshape(n, heads, dim)[on]
        at = (slots[on] // page, slice(None), slots[on] % page)
        if kind == "i8":
            code, step = quantised(val)
            want[x][at] = code.to(torch.int8)
            want_s[x][at] = step.float()
        else:
            want[x][at] = val
    kv.append(n, slots.data_ptr(), rows["k"].data_ptr(), 0 if shared else rows["v"].data_ptr(), wide.stride(0), wide.stride(0))
    kv.sync()
    for x in names:
        assert torch.equal(pools[x], want[x]), x
        if scales:  # one fp32 division of an fp32 maximum: half a step of it
            assert bool(((scales[x].double() - want_s[x].double()).abs() <= want_s[x].double() * 2.0 ** -23).all())
    if layout == "gaps":  # the values between rows
        base = pools["k"]._base
        assert not bool(base[..., dim:].any()) and not bool(base[:, :, page].any())


def test_append_of_more_tokens_than_one_round_of_indices():
    import torch
    n, page = 2 ** 18 + 77, 64
    c = Cache([0], 1, 32, page, "bf16", shared=True, spare=n // page + 2)
    c.k.zero_()
    rows = torch.randn((n, 1, 32), device="cuda").to(torch.bfloat16)
    slots = torch.randperm(c.n_pages * page, device="cuda")[:n]
    want = torch.zeros_like(c.k)
    want[slots // page, :, slots % page] = rows
    kv = c.handle(1)
    kv.append(n, slots.data_ptr(), rows.data_ptr())
    kv.sync()
    assert torch.equal(c.k, want)


def test_append_of_tiny_rows_to_eight_bits():
    """Rows of the smallest normal and subnormal values: their codes and scales like any others'."""
    import torch
    c = Cache([0], 1, 64, 16, "bf16", "i8", shared=True)
    rows = torch.randn((6, 1, 64), device="cuda").double() * torch.tensor([2.0 ** -126, 2.0 ** -128, 2.0 ** -132, 2.0 ** -60, 2.0 ** -61, 2.0 ** 100],
                                                                           dtype=torch.float64, device="cuda")[:, None, None]
    rows = rows.to(torch.bfloat16)
    slots = torch.arange(6, device="cuda")
    kv = c.handle(1)
    kv.append(6, slots.data_ptr(), rows.data_ptr())
    kv.sync()
    code, step = quantised(rows)
    assert torch.equal(c.k[0, :, :6].transpose(0, 1).double(), code)
    # the scale's division by 127: half a step of fp32, or of its smallest subnormal
    assert bool(((c.k_scale[0, :, :6].T.double() - step).abs() <= step * 2.0 ** -24 + 2.0 ** -150).all())


def test_append_reports_slots_outside_the_pool():
    import torch
    c = Cache([0], 2, 64, 16, spare=4)
    c.k.zero_()
    c.v.zero_()
    kv = c.handle(2)
    rows = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (64, 2 ** 40, 2 ** 62):
        slots = dev([3, bad, -7, 17], "int64")
        kv.append(4, slots.data_ptr(), rows.data_ptr(), rows.data_ptr())
        assert kv.sync(check=False) == 3 and "slot" in kv.last_error()
    assert float(c.k.float().sum()) == 2 * 2 * 64 and bool((c.k[0, :, 3] == 1).all()) and bool((c.v[1, :, 1] == 1).all())
    kv.append(0, 0, 0, 0)
    kv.sync()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_of_rows_that_are_no_numbers(bad):
    import torch
    c = Cache([16], 1, 32, 16, "bf16", "i8")
    rows = torch.ones((2, 32), dtype=torch.bfloat16, device="cuda")
    rows[1, 7] = bad
    slots = dev([int(c.table[0, 0]) * 16 + i for i in range(2)], "int64")
    kv = c.handle(1)
    kv.append(2, slots.data_ptr(), rows.data_ptr(), rows.data_ptr())
    kv.sync()
    s = c.v_scale[c.table[0, 0].long(), 0]
    assert math.isfinite(float(s[0])) and not math.isfinite(float(s[1]))
    q, out = torch.ones((1, 32), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 32), dtype=torch.bfloat16, device="cuda")
    kv.attend(1, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr())
    kv.sync()
    assert bool(torch.isnan(out).all())


def test_append_refusals():
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache([0], 2, 64, 16)
    one = Cache([0], 2, 64, 16, shared=True)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    s, p = dev([0] * 4, "int64").data_ptr(), x.data_ptr()
    ok = dict(n_tok=2, slots=s, k=p, v=p)
    for st, change in ((2, dict(n_tok=-1)), (2, dict(n_tok=2 ** 31)), (1, dict(slots=0)), (1, dict(k=0)), (1, dict(v=0)), (1, dict(k_stride=120)),
                       (1, dict(v_stride=130)), (1, dict(k=p + 2)), (1, dict(v=p + 8))):
        with pytest.raises(cvr.CvrError) as e:
            c.handle(2).append(**{**ok, **change})
        assert e.value.status == st, change
    with pytest.raises(cvr.CvrError):
        one.handle(2).append(**ok)
    with pytest.raises(cvr.CvrError):
        cvr.KvCache(cvr.make_kv_config(2, 2, 64, 16, 10, 2, 4)).append(**ok)


# ---- together ----
@pytest.mark.parametrize("cache,dtype,window,layout", [("same", "bf16", 0, "page"), ("i8", "f16", 0, "token"), ("same", "f16", 50, "gaps")])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps(cache, dtype, window, layout, captured):
    """A prompt of each request, then steps of one token, on one stream; page counts and the list's head stay on the
    device, in two sets of arrays that take turns. Captured, the three calls of a step are one graph per set."""
    import torch
    n, heads, group, dim, page, steps = 5, 2, 4, 64, 8, 12
    prompt = [0, 1, 7, 8, 30]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Cache([0] * n, heads, dim, page, dtype, cache, layout, max_pages=8, spare=60, seed=3)
        for x in (c.k_scale, c.v_scale):
            if x is not None:
                x.fill_(math.nan)
        kv = c.handle(heads * group, window, s.cuda_stream)
        free = torch.randperm(60, device="cuda").to(torch.int32)
        held, head = [dev([0] * n), dev([0] * n)], [dev([0]), dev([0])]
        hist = [[torch.zeros((0, heads, dim), dtype=torch.float64, device="cuda") for _ in range(n)] for _ in range(2)]
        slots, t_len, t_new = torch.empty((64,), dtype=torch.int64, device="cuda"), c.lens, dev([0] * n)
        rows = [torch.zeros((64, heads, dim), dtype=torch_type(dtype), device="cuda") for _ in range(2)]
        q, out = torch.zeros((n, heads * group, dim), dtype=torch_type(dtype), device="cuda"), torch.zeros((n, heads * group, dim), dtype=torch_type(dtype), device="cuda")
    torch.cuda.synchronize()
    graphs = [None, None]

    def calls(turn):
        kv.tables(n, t_len.data_ptr(), c.table.data_ptr(), t_new.data_ptr(), held[turn].data_ptr(), free.data_ptr(), 60, head[turn].data_ptr(),
                  held[1 - turn].data_ptr(), head[1 - turn].data_ptr(), slots.data_ptr(), 64)
        kv.append(64, slots.data_ptr(), rows[0].data_ptr(), rows[1].data_ptr())
        kv.attend(n, q.data_ptr(), t_len.data_ptr(), c.table.data_ptr(), 0.125, out.data_ptr())

    if captured:
        for turn in range(2):
            graphs[turn] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[turn], stream=s):
                calls(turn)
    lens, used = [0] * n, 0
    for step in range(steps):
        new = prompt if step == 0 else [1 if (step + r) % 4 else 0 for r in range(n)]
        lens = [a + b for a, b in zip(lens, new)]
        with torch.cuda.stream(s):
            t_len.copy_(dev(lens))
            t_new.copy_(dev(new))
            for x in rows:
                x.copy_(torch.randn(x.shape, device="cuda"))
            q.copy_(torch.randn(q.shape, device="cuda"))
            at = 0
            for r in range(n):
                for w in range(2):
                    val = rows[w][at:at + new[r]]
                    if cache == "i8":
                        code, st = quantised(val)
                        val = code * st.float().double()[..., None]
                    hist[w][r] = torch.cat([hist[w][r], val.double()])
                at += new[r]
            if captured:
                graphs[step % 2].replay()
            else:
                calls(step % 2)
        kv.sync()
        c.lens_list = lens
        ref, _, b_out, _ = c.reference(q, 0.125, window)
        assert_within(out, ref, b_out, f"step {step}")
        for r in range(n):  # the cache holds exactly the history
            for h in range(heads):
                for got, want in zip(c.rows(r, h, 0, lens[r]), (hist[0][r][:, h], hist[1][r][:, h])):
                    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -22).all()) if cache == "i8" else torch.equal(got, want)
        used = sum(-(-x // page) for x in lens)
        assert int(head[1 - step % 2]) == used and held[1 - step % 2].tolist() == [-(-x // page) for x in lens]
    assert used > n


def test_attend_is_the_scoring_paths_cross_attention():
    """The encoded histories of cvr_score, stored in pages with K = V, and its queries with its temperature: every
    candidate's attention over its request's pages is the decoded token that cvr_score made, up to both roundings to bf16."""
    import numpy as np
    import torch
    import cvr_ranking_model_gb300 as cvr
    import synth
    from gpu_util import GpuRun
    wl = synth.make_workload("tiny", n_req=5, cand_per_req=[1, 70, 3, 64, 9], seq_len=(3, 70, 129), user_rows=5000, item_rows=3000)
    g = GpuRun(wl, synth.make_weights(wl.n_layers, wl.seed, bias_scale=0.02), debug=False)
    g.run()
    L, R, B, page = wl.seq_len, wl.n_req, wl.n_cand, 16
    hs = torch.from_numpy(g.stage(cvr.STAGE_H, (R * sum(L), 128), torch.bfloat16)).cuda()
    z = torch.from_numpy(g.stage(cvr.STAGE_Z, (B, 16, 128), torch.bfloat16)).cuda()
    q = torch.from_numpy(g.stage(cvr.STAGE_Q, (B, 3, 128), torch.bfloat16)).cuda()
    req = torch.from_numpy(np.ascontiguousarray(wl.req_ids)).cuda().long()
    for grp in range(3):
        n = L[grp]
        states = hs[R * sum(L[:grp]):][:R * n].reshape(R * n, 4, 32)
        c = Cache([n] * R, 4, 32, page, "bf16", shared=True, seed=grp)
        c.k.fill_(math.nan)
        kv = c.handle(4, max_req=B)
        free, head = torch.randperm(c.n_pages, device="cuda").to(torch.int32), dev([0, 0])
        slots = torch.empty((R * n,), dtype=torch.int64, device="cuda")
        kv.tables(R, c.lens.data_ptr(), c.table.data_ptr(), c.lens.data_ptr(), free_pages=free.data_ptr(), n_free=c.n_pages,
                  slots=slots.data_ptr(), n_slots=R * n)
        rows = states.to(torch.bfloat16).contiguous()
        kv.append(R * n, slots.data_ptr(), rows.data_ptr())
        cand_table, cand_lens = c.table[req].contiguous(), c.lens[req].contiguous()
        qg, out = q[:, grp].to(torch.bfloat16).contiguous(), torch.empty((B, 128), dtype=torch.bfloat16, device="cuda")
        kv.attend(B, qg.data_ptr(), cand_lens.data_ptr(), cand_table.data_ptr(), 1.0 / (2.0 * 32 ** 0.5), out.data_ptr())
        kv.sync()
        want = z[:, 13 + grp]
        # cvr_score rounds its weights p to bf16 (2^-8 of sum p |v|, at most max |v|); both round their outputs
        big = states.reshape(R, n, 128).abs().amax(1)[req]
        assert bool(((out.double() - want).abs() <= 2 * 2.0 ** -8 * want.abs() + 2.0 ** -8 * big + 2.0 ** -12 * big).all())
