"""Calls of the paged history cache as a program may make them: without waits between them, while streams capture, with
arrays that overlap or are not aligned, with very many requests."""
import math

import pytest

from kv_util import Cache, assert_within, torch_type

pytestmark = pytest.mark.gpu


def dev(x, kind="int32"):
    import torch
    return torch.tensor(x, dtype=getattr(torch, kind), device="cuda")


@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("i8", "f16")])
def test_a_chain_of_calls_without_a_wait(cache, dtype):
    """Steps of tables, append and attend directly behind one another, each step with arrays of its own: every kernel starts
    while the ones before it still write what it reads."""
    import torch
    n, heads, group, dim, page, steps = 9, 2, 2, 64, 8, 40
    c = Cache([0] * n, heads, dim, page, dtype, cache, max_pages=16, spare=n * 16, seed=5)
    for x in (c.k_scale, c.v_scale):
        if x is not None:
            x.fill_(math.nan)
    lens = [[r + s * (r + 1) // 9 for r in range(n)] for s in range(steps)]
    new = [[b if s == 0 else b - a for a, b in zip(lens[s - 1], lens[s])] for s in range(steps)]
    most = max(sum(x) for x in new)
    t_lens, t_new = dev(lens), dev(new)
    rows = torch.randn((steps, 2, most, heads, dim), generator=c.gen, device="cuda").to(torch_type(dtype))
    q = torch.randn((steps, n, heads * group, dim), generator=c.gen, device="cuda").to(torch_type(dtype))
    free = torch.randperm(c.n_pages, device="cuda").to(torch.int32)
    results = []
    for waits in (False, True, False):
        held, head = torch.zeros((steps + 1, n), dtype=torch.int32, device="cuda"), torch.zeros(steps + 1, dtype=torch.int32, device="cuda")
        slots, out = torch.zeros((steps, most), dtype=torch.int64, device="cuda"), torch.zeros_like(q)
        c.table.fill_(-1)
        torch.cuda.synchronize()
        kv = c.handle(heads * group)
        for s in range(steps):
            kv.tables(n, t_lens[s].data_ptr(), c.table.data_ptr(), t_new[s].data_ptr(), held[s].data_ptr(), free.data_ptr(), c.n_pages,
                      head[s:].data_ptr(), held[s + 1].data_ptr(), head[s + 1:].data_ptr(), slots[s].data_ptr(), most)
            if waits:
                kv.sync()
            kv.append(most, slots[s].data_ptr(), rows[s, 0].data_ptr(), rows[s, 1].data_ptr())
            if waits:
                kv.sync()
            kv.attend(n, q[s].data_ptr(), t_lens[s].data_ptr(), c.table.data_ptr(), 0.125, out[s].data_ptr())
            if waits:
                kv.sync()
        kv.sync()
        results.append((held, head, slots, out, c.table.clone()))
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))
    c.lens_list = lens[-1]
    ref, _, bound, _ = c.reference(q[-1], 0.125)
    assert_within(results[0][3][-1], ref, bound, "out")


def small(seed, q_heads=8):
    import torch
    c = Cache([300, 20], 2, 64, 16, "bf16", seed=seed)
    q = torch.randn((2, q_heads, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
    return c, q, torch.zeros_like(q)


def attend(kv, c, q, out):
    kv.attend(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr())


def check(c, q, out):
    ref, _, bound, _ = c.reference(q, 0.1)
    assert_within(out, ref, bound, "out")


def test_a_handle_of_another_stream_while_a_stream_captures():
    """A handle may be made, used, waited for and destroyed on a stream of its own while another stream captures in the default
    (global) mode, and the capture goes on."""
    import torch
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    c, q, out = small(1)
    out2 = torch.zeros_like(out)
    kv = c.handle(8, stream=s.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attend(kv, c, q, out)
        kv2 = c.handle(8, stream=other.cuda_stream)
        attend(kv2, c, q, out2)
        kv2.sync()
        kv2.close()
        attend(kv, c, q, out)
    check(c, q, out2)
    with torch.cuda.stream(s):
        graph.replay()
    kv.sync()
    check(c, q, out)


def test_sync_of_a_stream_that_captures_is_refused():
    import torch
    import cvr_ranking_model_gb300 as cvr
    s = torch.cuda.Stream()
    c, q, out = small(2)
    kv = c.handle(8, stream=s.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attend(kv, c, q, out)
        with pytest.raises(cvr.CvrError) as e:
            kv.sync()
    assert e.value.status == 1 and "captur" in str(e.value)
    with torch.cuda.stream(s):
        graph.replay()
    kv.sync()
    check(c, q, out)


def test_the_legacy_stream_is_refused_while_a_blocking_stream_captures():
    """A blocking stream's capture makes the legacy default stream unusable: a handle is not made on it or waited for, and the
    capture goes on."""
    import ctypes
    import torch
    import cvr_ranking_model_gb300 as cvr
    raw = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(raw))) == 0
    s = torch.cuda.ExternalStream(raw.value)
    c, q, out = small(3)
    kv, legacy = c.handle(8, stream=s.cuda_stream), c.handle(8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s, capture_error_mode="relaxed"):
        with pytest.raises(cvr.CvrError) as made:
            c.handle(8)
        with pytest.raises(cvr.CvrError) as waited:
            legacy.sync()
        attend(kv, c, q, out)
    assert made.value.status == 1 and waited.value.status == 1
    with torch.cuda.stream(s):
        graph.replay()
    kv.sync()
    check(c, q, out)
    kv.close()
    torch.cuda.synchronize()
    del graph
    assert int(torch.cuda.cudart().cudaStreamDestroy(raw.value)) == 0


def refused(call, **args):
    import cvr_ranking_model_gb300 as cvr
    with pytest.raises(cvr.CvrError) as e:
        call(**args)
    assert e.value.status == 1, args


def test_arrays_that_are_not_aligned_are_refused():
    import torch
    c, q, out = small(4)
    kv = c.handle(8)
    x = torch.zeros(4096, dtype=torch.int64, device="cuda")
    p = x.data_ptr()
    ok = dict(n_req=2, lens=p, table=p + 256, new_lens=p + 512, held=p + 768, free_pages=p + 1024, n_free=8, free_head=p + 1280, pages=p + 1536,
              free_head_out=p + 1792, slots=p + 2048, n_slots=4)
    for name in ("lens", "table", "new_lens", "held", "free_pages", "free_head", "pages", "free_head_out"):
        for by in (1, 2, 3):
            refused(kv.tables, **{**ok, name: ok[name] + by})
    for by in (1, 2, 4):
        refused(kv.tables, **{**ok, "slots": ok["slots"] + by})
        refused(kv.append, n_tok=1, slots=p + by, k=q.data_ptr(), v=q.data_ptr())
    ok = dict(n_req=2, q=q.data_ptr(), lens=c.lens.data_ptr(), table=c.table.data_ptr(), scale=0.1, out=out.data_ptr(), lse=p)
    for name in ("lens", "table", "lse"):
        for by in (1, 2, 3):
            refused(kv.attend, **{**ok, name: ok[name] + by})
    kv.attend(**ok)
    kv.sync()
    check(c, q, out)


def test_arrays_that_overlap_are_refused():
    """Whatever a call writes lies apart from all that it reads or writes, wholly and in part; neighbours are fine."""
    import torch
    c, _, _ = small(5)
    kv = c.handle(8)
    n, cols = 2, c.max_pages
    x = torch.zeros(4096, dtype=torch.int32, device="cuda")
    p = x.data_ptr()
    size = dict(lens=n, new_lens=n, held=n, free_pages=7, free_head=1, table=n * cols, pages=n, free_head_out=1, slots=2 * 4)
    at, ok = 0, dict(n_req=n, n_free=7, n_slots=4)
    for name, words in size.items():
        if name == "slots":
            at += at % 2
        ok[name] = p + 4 * at
        at += words
    written = ("table", "pages", "free_head_out", "slots")
    for one in written:
        for other in size:
            if other == one:
                continue
            first, last = ok[other], ok[other] + 4 * (size[other] - 1)
            starts = {first, last, first - 4 * (size[one] - 1), last - 4 * (size[one] - 1)}
            for s in starts:
                if one != "slots" or s % 8 == 0:
                    refused(kv.tables, **{**ok, one: s})
    x[0:2] = dev([4, 0])
    x[2:4] = dev([4, 0])
    x[6:13] = dev([3, 4, 5, 6, 7, 8, 9])
    kv.tables(**ok)
    kv.sync()
    assert x[:4].tolist() == [4, 0, 4, 0] and x[14:16].tolist() == [3, 0] and x[(ok["pages"] - p) // 4:][:3].tolist() == [1, 0, 1]
    assert x[(ok["slots"] - p) // 4:][:10:2].tolist() == [48, 49, 50, 51, 0]


@pytest.mark.parametrize("n,cols", [(42000, 65536), (500, 2 ** 23)])
def test_more_fresh_entries_than_32_bit_sums_hold(n, cols):
    """A table above 8 GB of which nearly every entry is fresh: those behind the free list's end are -1 to the last one."""
    import torch
    import cvr_ranking_model_gb300 as cvr
    n_free, page = 600_001, 8
    kv = cvr.KvCache(cvr.make_kv_config(1, 1, 32, page, n_free, n, cols))
    lens = torch.full((n,), cols * page, dtype=torch.int32, device="cuda")
    held = (torch.arange(n, device="cuda") % 3 == 0).to(torch.int32)
    table = torch.full((n, cols), 77, dtype=torch.int32, device="cuda")
    free = torch.randperm(n_free, device="cuda").to(torch.int32)
    pages, head, none = torch.empty_like(held), dev([0]), torch.zeros_like(held)
    kv.tables(n, lens.data_ptr(), table.data_ptr(), new_lens=none.data_ptr(), held=held.data_ptr(), free_pages=free.data_ptr(),
              n_free=n_free, pages=pages.data_ptr(), free_head_out=head.data_ptr())
    assert kv.sync(check=False) == 8 and int(head) == n_free and int(pages.sum()) == n_free + int(held.sum())
    assert bool((table[::3, 0] == 77).all())
    table[::3, 0] = -1
    rows = 3 + n_free // cols  # the rows that hold pages
    flat = table[:rows].flatten()
    assert torch.equal(flat[flat != -1], free) and int(flat.max()) == n_free - 1
    for a in range(rows, n, 2000):
        assert int(table[a:a + 2000].max()) == -1 and int(table[a:a + 2000].min()) == -1
    with pytest.raises(cvr.CvrError) as e:
        kv.tables(n, lens.data_ptr(), table.data_ptr(), free_pages=free.data_ptr(), n_free=2 ** 31 - 1)
    assert e.value.status == 2


@pytest.mark.parametrize("cache", ["same", "i8"])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 161, 2 ** 31 - 1])
def test_a_length_out_of_range_is_reported_and_used_clamped(cache, bad):
    import torch
    c = Cache([160, 30], 2, 64, 16, "bf16", cache, seed=6, max_pages=10)
    kv = c.handle(8)
    q = torch.randn((2, 8, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((2, 8), 7.0, device="cuda")
    c.lens[0] = c.lens_list[0] = bad
    kv.attend(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr(), lse.data_ptr())
    assert kv.sync(check=False) == 6 and "length" in kv.last_error()
    ref, ref_lse, bound, b_lse = c.reference(q, 0.1)  # (of no token, or of max_pages * page_size)
    assert_within(out, ref, bound, "out")
    assert_within(lse, ref_lse, b_lse, "lse")


@pytest.mark.parametrize("n", [20000, 65535])
@pytest.mark.parametrize("dtype,cache,heads,group,dim,window", [("bf16", "same", 1, 2, 32, 0), ("f16", "i8", 2, 1, 64, 9), ("bf16", "i8", 1, 17, 32, 0)])
def test_very_many_requests_with_histories(n, dtype, cache, heads, group, dim, window):
    """Tens of thousands of requests of 0 to 24 tokens; the bounds as in Cache.reference, for all requests at once."""
    import torch
    import cvr_ranking_model_gb300 as cvr
    from kv_util import EPS, cvr_type
    page, cols = 8, 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + dim)
    lens = torch.randint(0, page * cols + 1, (n,), generator=gen, device="cuda").to(torch.int32)
    table = torch.randperm(n * cols, generator=gen, device="cuda").to(torch.int32).view(n, cols)
    x = [torch.randn((n * cols, heads, page, dim), generator=gen, device="cuda") for _ in range(2)]
    scale = [None, None]
    if cache == "i8":
        x = [(t * 40).round().clamp(-127, 127).to(torch.int8) for t in x]
        scale = [torch.rand((n * cols, heads, page), generator=gen, device="cuda") * 0.05 for _ in range(2)]
    else:
        x = [t.to(torch_type(dtype)) for t in x]
    q = torch.randn((n, heads * group, dim), generator=gen, device="cuda").to(torch_type(dtype))
    out, lse = torch.full_like(q, 7.0), torch.full((n, heads * group), 7.0, device="cuda")
    torch.cuda.synchronize()
    kv = cvr.KvCache(cvr.make_kv_config(heads * group, heads, dim, page, n * cols, n, cols, cvr_type(dtype), cvr_type("i8" if cache == "i8" else dtype),
                                        window, x[0].data_ptr(), k_scale=scale[0].data_ptr() if scale[0] is not None else 0,
                                        v=x[1].data_ptr(), v_scale=scale[1].data_ptr() if scale[1] is not None else 0))
    kv.attend(n, q.data_ptr(), lens.data_ptr(), table.data_ptr(), dim ** -0.5, out.data_ptr(), lse.data_ptr())
    kv.sync()
    for a in range(0, n, 8192):
        r = slice(a, min(a + 8192, n))
        k, v = ((t[table[r].long()].double() * (1.0 if s is None else s[table[r].long()].double()[..., None])).transpose(1, 2).flatten(2, 3)
                for t, s in zip(x, scale))  # [request, head, token, dim]
        j, m = torch.arange(page * cols, device="cuda"), lens[r].long()[:, None]
        seen = ((j < m) & (j >= (m - window if window else 0)))[:, None, None, :]
        y = q[r].double().unflatten(1, (heads, group))
        s = torch.where(seen, y @ k.transpose(2, 3) * dim ** -0.5, -math.inf)
        p = torch.nan_to_num(torch.softmax(s, 3), nan=0.0)
        o, size = p @ v, p @ v.abs()
        top = torch.where(seen, (y.abs() @ k.abs().transpose(2, 3)) * dim ** -0.5, 0.0).amax(3, keepdim=True)
        rel = top * dim * 2.0 ** -23 + torch.where(seen, s.abs(), 0.0).amax(3, keepdim=True) * 2.0 ** -22 + 2.0 ** -21
        sums = (page * cols / 16 + 64) * 2.0 ** -23
        assert_within(out[r], o.flatten(1, 2), (EPS[dtype] * o.abs() + (2 * (rel + 2.0 ** -15) + 2 * sums) * size + 2.0 ** -25).flatten(1, 2), "out")
        want = torch.logsumexp(s, 3)
        assert_within(lse[r], want.flatten(1, 2), (rel[..., 0] + sums + torch.where(torch.isinf(want), 0.0, want.abs()) * 2.0 ** -22).flatten(1, 2), "lse")
