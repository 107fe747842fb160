"""cvr_kv_attend against its definition in 64 bits: head layouts, lengths around every block size, types, pool layouts,
windows, empty rows; rubbish in every place that must not be read; its refusals and device-side errors."""
import math

import pytest

from kv_util import Cache, assert_within, torch_type

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]


def attend(c, q_heads, window=0, scale=None, seed=1, gain=1.0, handle=None):
    """One call with gaps between the rows of q and out and rows behind the last; checks what must stay as it was."""
    import torch
    n = len(c.lens_list)
    scale = c.dim ** -0.5 if scale is None else scale
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q = torch.full((n, q_heads * c.dim + 8), math.nan, dtype=torch_type(c.dtype), device="cuda")
    q[:, :q_heads * c.dim] = (torch.randn((n, q_heads * c.dim), generator=gen, device="cuda") * gain).to(q.dtype)
    out = torch.full((n + 2, q_heads * c.dim + 16), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n + 2, q_heads), 7.0, device="cuda")
    kv = handle or c.handle(q_heads, window)
    kv.attend(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, out.data_ptr(), lse.data_ptr(), q.stride(0), out.stride(0))
    st = kv.sync(check=False)
    assert bool((out[n:] == 7).all()) and bool((out[:, q_heads * c.dim:] == 7).all()) and bool((lse[n:] == 7).all())
    return q[:, :q_heads * c.dim].reshape(n, q_heads, c.dim), out[:n, :q_heads * c.dim].reshape(n, q_heads, c.dim), lse[:n], st


def check(c, q_heads, window=0, scale=None, **kw):
    scale = c.dim ** -0.5 if scale is None else scale
    q, out, lse, st = attend(c, q_heads, window, scale, **kw)
    assert st == 0
    ref, ref_lse, b_out, b_lse = c.reference(q, scale, window)
    assert_within(lse, ref_lse, b_lse, "lse")
    assert_within(out, ref, b_out, "out")
    return out, lse


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "i8"), ("f16", "i8")])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("heads,group", [(4, 1), (2, 4), (1, 17), (1, 64)])
def test_types_dims_and_heads(dtype, cache, dim, heads, group):
    check(Cache(EDGES, heads, dim, 16, dtype, cache, seed=dim + group), heads * group)


@pytest.mark.parametrize("layout", ["page", "token", "gaps"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,cache", [(32, "same"), (64, "i8"), (128, "same"), (32, "i8"), (128, "i8"), (64, "same")])
def test_pages_and_pool_layouts(layout, page, dim, cache):
    check(Cache([300, 0, 1, page - 1, page, page + 1, 777], 3, dim, page, "bf16", cache, layout, seed=page), 6)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 15, 16, 31, 32, 33, 48, 63])
def test_group_sizes(group):
    check(Cache([70, 1, 200], 2, 64, 16, "f16", seed=group), 2 * group)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("dim,page,cache", [(32, 8, "same"), (128, 16, "same"), (64, 64, "i8"), (128, 256, "i8")])
def test_windows(window, dim, page, cache):
    check(Cache([0, 1, 16, 17, 65, 130, 999, 1500], 2, dim, page, "bf16", cache, "token", seed=window % 97), 8, window)


@pytest.mark.parametrize("dtype,cache,dim,group", [("bf16", "same", 32, 1), ("f16", "same", 128, 4), ("bf16", "i8", 64, 16), ("f16", "i8", 32, 33)])
def test_one_pool_for_keys_and_values(dtype, cache, dim, group):
    check(Cache(EDGES, 4, dim, 32, dtype, cache, shared=True, seed=5), 4 * group)


@pytest.mark.parametrize("n,heads,group,dim", [(70001, 1, 1, 32), (40000, 1, 8, 128), (20001, 8, 4, 128), (30000, 2, 64, 64), (50001, 1, 16, 64),
                                              (30000, 1, 32, 128), (40000, 1, 64, 32)])
@pytest.mark.parametrize("cache", ["same", "i8"])
def test_long_histories_split_over_the_gpu(n, heads, group, dim, cache):
    check(Cache([n], heads, dim, 64, "bf16", cache, seed=n), heads * group)


def test_ragged_batch_long_and_short():
    check(Cache([5000, 1, 0, 0, 64, 12345, 3, 700] + [0] * 40 + [9] * 30, 2, 128, 16, "f16", seed=3), 8)


@pytest.mark.parametrize("tokens", [30000, 60000, 90000, 130000, 200000, 400000])
@pytest.mark.parametrize("dim,heads,group,cache", [(128, 2, 4, "same"), (64, 2, 16, "i8"), (32, 4, 1, "same"), (128, 1, 24, "i8")])
def test_runs_of_every_length(tokens, dim, heads, group, cache):
    """Uneven requests, empty ones among them, over runs from two tiles to many."""
    share = [0, 1, 0.2, 130, 3, 2.1, 0, 0.7, 5, 63]
    lens = [int(tokens / heads * x / sum(share)) for x in share] + [1, 129, 0]
    check(Cache(lens, heads, dim, 64, "bf16", cache, seed=tokens), heads * group)


def test_many_short_requests():
    lens = [(i * 37) % 23 for i in range(3000)]
    check(Cache(lens, 1, 32, 8, "bf16", seed=4), 2)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 40.0])
@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("bf16", "i8"), ("f16", "i8")])
def test_scales(scale, dtype, cache):
    check(Cache([1, 50, 333], 2, 64, 16, dtype, cache, seed=8), 4, scale=scale)


@pytest.mark.parametrize("cache", ["same", "i8"])
@pytest.mark.parametrize("log2_q,log2_k,scale", [(126, -90, 2.0 ** -38), (124, -90, 2.0 ** -36), (-130, 100, 2.0 ** 28), (-126, 100, 2.0 ** 24)])
def test_queries_at_the_ends_of_bf16(log2_q, log2_k, scale, cache):
    c = Cache([1, 50, 333], 2, 64, 16, "bf16", cache, seed=22)
    for r, n in enumerate(c.lens_list):
        p = c.table[r, :-(-n // 16)].long()
        if cache == "i8":
            c.k_scale[p] *= 2.0 ** log2_k
        else:
            c.k[p] = (c.k[p].float() * 2.0 ** log2_k).to(c.k.dtype)  # (exact: powers of two, far from the type's ends)
    check(c, 4, scale=scale, gain=0.9 * 2.0 ** log2_q)


def test_twelve_thousand_requests_most_of_them_empty():
    check(Cache([3 if i % 7 == 0 else 40 if i == 11999 else 0 for i in range(12000)], 1, 32, 8, "f16", seed=18), 1)


def test_keys_and_values_laid_out_differently():
    """Keys page by page and head by head, values token by token; then both in one tensor, page by page."""
    import torch
    c = Cache([300, 5, 64], 2, 64, 16, "bf16", seed=19)
    v = torch.empty((c.n_pages, 16, 2, 64), dtype=c.v.dtype, device="cuda").permute(0, 2, 1, 3)
    v.copy_(c.v)
    c.v = v
    check(c, 8)
    both = torch.empty((c.n_pages, 2, 2, 16, 64), dtype=c.v.dtype, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    c.k, c.v = both[:, 0], both[:, 1]
    check(c, 8)


def test_a_pool_of_one_page_and_one_head():
    """Strides of dimensions of one row are not used, whatever they are."""
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache([13], 1, 32, 16, "f16", seed=20, spare=0)
    cfg = cvr.make_kv_config(3, 1, 32, 16, 1, 1, c.max_pages, cvr.DTYPE_F16, k=c.k.data_ptr(), k_strides=(0, -7, 32), v=c.v.data_ptr(),
                             v_strides=(-1, 0, 32))
    check(c, 3, handle=cvr.KvCache(cfg))


def test_row_scales_of_either_sign():
    import torch
    c = Cache([100, 7], 2, 32, 16, "bf16", "i8", seed=21)
    for s in (c.k_scale, c.v_scale):
        s.mul_(torch.where(torch.rand(s.shape, generator=c.gen, device="cuda") < 0.5, -1.0, 1.0))
    check(c, 4)


@pytest.mark.parametrize("cache", ["same", "i8"])
def test_large_logits_pick_one_token(cache):
    check(Cache([40, 500], 2, 128, 16, "f16", cache, seed=9, spread=3.0), 4, scale=1.0, gain=20.0)


def test_row_scales_of_very_different_size():
    """Rows whose scales lie far apart, tiny and zero ones among them: each weighs as its value."""
    import torch
    c = Cache([300, 65, 1], 2, 64, 16, "f16", "i8", seed=10)
    for s in (c.k_scale, c.v_scale):
        e = torch.randint(-20, 3, s.shape, generator=c.gen, device="cuda")
        s.mul_(torch.exp2(e.float()))
    c.v_scale[torch.rand(c.v_scale.shape, generator=c.gen, device="cuda") < 0.2] = 0.0
    c.v_scale[c.table[2, 0].long()] = 0.0
    check(c, 8)


def test_the_same_bits_on_every_call():
    import torch
    c = Cache([30000, 11, 2000], 2, 128, 32, "bf16", seed=11)
    kv = c.handle(8)
    first = attend(c, 8, handle=kv)
    for _ in range(5):
        again = attend(c, 8, handle=kv)
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_pool_larger_than_32_bit_offsets():
    """More than 2^32 values: rows at both ends of the pool."""
    import torch
    c = Cache([100, 70], 1, 128, 256, "bf16", shared=True, seed=12, spare=2 ** 32 // (256 * 128) + 10)
    assert c.k.numel() > 2 ** 32
    ids = torch.tensor([[c.n_pages - 1], [0]], dtype=torch.int32, device="cuda")
    for r in range(2):
        c.k[ids[r, 0].long()].copy_(torch.randn((1, 256, 128), generator=c.gen, device="cuda").to(c.k.dtype))
    c.table[:, :1] = ids
    check(c, 4)


def test_pages_shared_between_requests():
    c = Cache([100, 100, 37], 2, 64, 16, "bf16", seed=13)
    c.table[1] = c.table[0]
    c.table[2] = c.table[0]
    check(c, 4)


def test_nothing_seen_and_no_request():
    import torch
    c = Cache([0, 0, 0], 2, 64, 16)
    _, out, lse, st = attend(c, 8)
    assert st == 0 and not bool(out.any()) and bool(torch.isneginf(lse).all())
    c.handle(8).attend(0, 0, 0, 0, 1.0, 0)


def test_lse_may_be_left_out():
    import torch
    c = Cache([100], 2, 64, 16)
    q = torch.randn((1, 4, 64), device="cuda").to(torch.bfloat16)
    out, out2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((1, 4), device="cuda")
    kv = c.handle(4)
    kv.attend(1, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr())
    kv.attend(1, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out2.data_ptr(), lse.data_ptr())
    kv.sync()
    assert torch.equal(out, out2)


def test_values_that_are_no_numbers_reach_the_output():
    import torch
    c = Cache([50, 50], 1, 32, 16, "bf16", seed=14)
    c.v[c.table[0, 1].long(), 0, 3, 5] = math.nan
    _, out, lse, st = attend(c, 2)
    assert st == 0 and bool(torch.isnan(out[0, :, 5]).all()) and bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse).all())
    assert int(torch.isnan(out).sum()) == 2
    c.k[c.table[1, 0].long(), 0, 0, 0] = math.nan
    _, out, lse, st = attend(c, 2)
    assert st == 0 and bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())


def test_bad_pages_and_lengths_are_reported_and_spare_the_others():
    import torch
    c = Cache([100, 100, 40, 9], 2, 64, 16, "bf16", seed=15)
    ref = c.handle(4)
    q, good, _, st = attend(c, 4, handle=ref)
    assert st == 0
    c.k[0].zero_()  # what a bad page reads instead
    c.v[0].zero_()
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = int(c.table[0, 2])
        c.table[0, 2] = bad
        _, out, _, st = attend(c, 4, handle=ref)
        assert st == 3 and "page" in ref.last_error()
        c.table[0, 2] = t
        same = [r for r in (1, 2, 3) if 0 not in c.table[r, :-(-c.lens_list[r] // 16)].tolist()]
        assert same and all(torch.equal(out[r], good[r]) for r in same)
    for bad in (-1, -2 ** 31, c.max_pages * 16 + 1, 2 ** 31 - 1):
        c.lens[3] = bad
        _, out, _, st = attend(c, 4, handle=ref)
        assert st in (3, 6)
        if bad < 0:
            assert st == 6 and not bool(out[3].any())
    c.lens[3] = 9
    assert attend(c, 4, handle=ref)[3] == 0 and ref.last_error() == ""


def test_capture_and_replay():
    import torch
    s = torch.cuda.Stream()
    c = Cache([3000, 20, 0, 129], 2, 128, 16, "bf16", seed=16)
    q = torch.randn((4, 8, 128), device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros((4, 8), device="cuda")
    torch.cuda.synchronize()
    kv = c.handle(8, stream=s.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(3):
            kv.attend(4, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr(), lse.data_ptr())
    for lens in ([3000, 20, 0, 129], [1, 0, 0, 64], [2999, 20, 0, 5]):
        c.lens_list = lens
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        kv.sync()
        ref, ref_lse, b_out, b_lse = c.reference(q, 0.1)
        assert_within(out, ref, b_out, "out")
        assert_within(lse, ref_lse, b_lse, "lse")


def test_no_handle_is_made_while_its_stream_captures():
    import torch
    import cvr_ranking_model_gb300 as cvr
    s = torch.cuda.Stream()
    c = Cache([300, 20], 2, 64, 16, "bf16", seed=24)
    q = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    kv = c.handle(8, stream=s.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s, capture_error_mode="relaxed"):
        with pytest.raises(cvr.CvrError) as e:
            c.handle(8, stream=s.cuda_stream)
        kv.attend(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr())
    assert e.value.status == 1
    with torch.cuda.stream(s):
        graph.replay()
    kv.sync()
    ref, _, b_out, _ = c.reference(q, 0.1)
    assert_within(out, ref, b_out, "out")


def test_two_handles_on_two_streams_at_once():
    import torch
    c = Cache([20000, 300, 7], 2, 128, 32, "bf16", seed=17)
    q = torch.randn((3, 8, 128), device="cuda").to(torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    kvs = [c.handle(8, stream=s.cuda_stream) for s in streams]
    for _ in range(20):
        for kv, out in zip(kvs, outs):
            kv.attend(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, out.data_ptr())
    for kv in kvs:
        kv.sync()
    ref, _, b_out, _ = c.reference(q, 0.1)
    for out in outs:
        assert_within(out, ref, b_out, "out")


def test_histories_too_long_together():
    """More tiles than a call can number: reported, nothing written but for the empty request, and the handle stays good."""
    import torch
    import cvr_ranking_model_gb300 as cvr
    k = torch.randn((1, 256, 256, 32), device="cuda").to(torch.bfloat16)
    kv = cvr.KvCache(cvr.make_kv_config(256, 256, 32, 256, 1, 4, 2 ** 22, k=k.data_ptr()))
    lens = torch.tensor([2 ** 30, 0, 2 ** 30, 2 ** 30], dtype=torch.int32, device="cuda")
    table = torch.zeros((4, 2 ** 22), dtype=torch.int32, device="cuda")
    q = torch.randn((4, 256, 32), device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    kv.attend(4, q.data_ptr(), lens.data_ptr(), table.data_ptr(), 0.1, out.data_ptr())
    assert kv.sync(check=False) == 2 and "too long together" in kv.last_error()
    assert bool((out[[0, 2, 3]] == 7).all()) and not bool(out[1].any())
    lens.copy_(torch.tensor([256, 0, 1, 100], dtype=torch.int32))
    kv.attend(4, q.data_ptr(), lens.data_ptr(), table.data_ptr(), 0.1, out.data_ptr())
    assert kv.sync(check=False) == 0 and torch.equal(out[2], k[0, :, 0])


def test_refusals():
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache([10, 10], 2, 64, 16)
    kv = c.handle(4)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    lens, table = c.lens.data_ptr(), c.table.data_ptr()
    ok = dict(n_req=2, q=q.data_ptr(), lens=lens, table=table, scale=1.0, out=q.data_ptr())
    for status, change in ((2, dict(n_req=3)), (2, dict(n_req=-1)), (1, dict(q=0)), (1, dict(lens=0)), (1, dict(table=0)), (1, dict(out=0)),
                           (1, dict(scale=math.nan)), (1, dict(scale=math.inf)), (1, dict(q=q.data_ptr() + 2)), (1, dict(out=q.data_ptr() + 8)),
                           (1, dict(q_stride=248)), (1, dict(q_stride=260)), (1, dict(out_stride=-256)), (1, dict(out_stride=258))):
        with pytest.raises(cvr.CvrError) as e:
            kv.attend(**{**ok, **change})
        assert e.value.status == status, change
    bare = cvr.KvCache(cvr.make_kv_config(4, 2, 64, 16, 10, 2, 4))
    with pytest.raises(cvr.CvrError) as e:
        bare.attend(**ok)
    assert e.value.status == 1
