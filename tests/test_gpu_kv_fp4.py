"""Pools of 4 bits: rows appended against the definition's exact quotients, rows read back, attention of one new token."""
import math

import pytest

from kv_more_util import EPS, Cache4, Pool4, quantised, value_of
from kv_util import assert_within, torch_type

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]


def attend(c, q_heads, window=0, scale=None, seed=1, gain=1.0):
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
    kv = c.handle(q_heads, window)
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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("heads,group", [(4, 1), (2, 4), (3, 3), (2, 7), (1, 8), (1, 12), (1, 17), (1, 64)])
def test_types_dims_and_heads(dtype, dim, heads, group):
    check(Cache4(EDGES, heads, dim, 16, dtype, seed=dim + group), heads * group)


@pytest.mark.parametrize("layout", ["page", "token", "gaps"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,group", [(32, 2), (64, 16), (128, 2), (128, 9), (128, 40)])
def test_pages_and_pool_layouts(layout, page, dim, group):
    check(Cache4([300, 0, 1, page - 1, page, page + 1, 777], 3, dim, page, "bf16", layout=layout, seed=page), 3 * group)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("dim,page", [(32, 8), (128, 16), (64, 64), (128, 256)])
def test_windows(window, dim, page):
    check(Cache4([0, 1, 16, 17, 65, 130, 999, 1500], 2, dim, page, "bf16", layout="token", seed=window % 97), 8, window)


@pytest.mark.parametrize("dtype,dim,group", [("bf16", 32, 1), ("f16", 128, 4), ("bf16", 64, 16), ("f16", 32, 33), ("bf16", 128, 64)])
def test_one_pool_for_keys_and_values(dtype, dim, group):
    check(Cache4(EDGES, 4, dim, 32, dtype, shared=True, seed=5), 4 * group)


@pytest.mark.parametrize("n,heads,group,dim", [(70001, 1, 1, 32), (40000, 1, 8, 128), (20001, 8, 4, 128), (30000, 2, 64, 64), (30000, 1, 32, 128)])
def test_long_histories_split_over_the_gpu(n, heads, group, dim):
    check(Cache4([n], heads, dim, 64, "bf16", seed=n), heads * group)


@pytest.mark.parametrize("tokens", [30000, 130000, 400000])
@pytest.mark.parametrize("dim,heads,group", [(128, 2, 4), (64, 2, 16), (32, 4, 1), (128, 1, 24)])
def test_runs_of_every_length(tokens, dim, heads, group):
    share = [0, 1, 0.2, 130, 3, 2.1, 0, 0.7, 5, 63]
    lens = [int(tokens / heads * x / sum(share)) for x in share] + [1, 129, 0]
    check(Cache4(lens, heads, dim, 64, "bf16", seed=tokens), heads * group)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 40.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales(scale, dtype):
    check(Cache4([1, 50, 333], 2, 64, 16, dtype, seed=8), 4, scale=scale)


@pytest.mark.parametrize("log2_q,log2_k,scale", [(126, -90, 2.0 ** -38), (-130, 100, 2.0 ** 28)])
def test_queries_at_the_ends_of_bf16(log2_q, log2_k, scale):
    c = Cache4([1, 50, 333], 2, 64, 16, "bf16", seed=22)
    c.k.scale.mul_(2.0 ** log2_k)
    check(c, 4, scale=scale, gain=0.9 * 2.0 ** log2_q)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [2, 6, 12, 24, 40])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("at", [[0], [150, 299]])
def test_a_large_value_without_weight_leaves_the_others_their_bits(dtype, group, dim, at):
    """Tokens whose V scale is far above the others', to which half of the query rows give a weight of about 2^-60 and the others nearly
    all of it. The bound is the one of values far apart: what vanishes is 2^-33 of the row's largest weight times V scale, times values of up
    to 2688, per token, and the split of a weight costs 2^-21."""
    import torch
    n = 300
    c = Cache4([n, 17], 2, dim, 16, dtype, seed=dim + group)
    q = torch.full((2, 2 * group, dim), 1.0, device="cuda")
    q[:, 1::2] = -1.0
    q += 0.01 * torch.randn(q.shape, generator=c.gen, device="cuda")
    q = q.to(torch_type(dtype))
    small, large = (-16, 24) if dtype == "bf16" else (-24, 1)
    for r in range(2):
        p = c.table[r, :-(-c.lens_list[r] // 16)].long()
        c.k.scale[p] = 2.0 ** -20
        c.v.scale[p] = 2.0 ** small
        c.v.block[p] = 0x38 + c.v.block[p] % 8  # 1 .. 1.875
    for j in at:
        p, i = int(c.table[0, j // 16]), j % 16
        c.k.codes[p, :, i] = 0xaa  # -1, -1
        c.k.block[p, :, i] = 0x38
        c.k.scale[p, :, i] = 1.0
        c.v.scale[p, :, i] = 2.0 ** large
    scale = 42.0 / dim
    out, lse = torch.zeros_like(q), torch.zeros((2, 2 * group), device="cuda")
    kv = c.handle(2 * group)
    kv.attend(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, out.data_ptr(), lse.data_ptr())
    kv.sync()
    ref, bound = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for r in range(2):
        for h in range(2):
            m = c.lens_list[r]
            k, v = c.rows(r, h, 0, m)
            j = torch.arange(m, device="cuda")
            vs = c.v.scale[c.table[r].long()[j // 16], h, j % 16].double()
            rows = slice(h * group, (h + 1) * group)
            x = q[r, rows].double()
            s = x @ k.T * scale
            p = torch.softmax(s, 1)
            o, size = p @ v, p @ v.abs()
            ref[r, rows] = o
            logit = (x.abs() @ k.abs().T * scale).amax(1, keepdim=True) * dim * 2.0 ** -23 + s.abs().amax(1, keepdim=True) * 4 * 2.0 ** -24
            logit = logit + x.abs().amax(1, keepdim=True) * k.abs().sum(1).amax() * scale * 2.0 ** -25  # (queries held in fp16)
            vanish = 2.0 ** -33 * 2688 * (p * vs).amax(1, keepdim=True) * m
            bound[r, rows] = EPS[dtype] * o.abs() + (2 * (logit + 2.0 ** -21 + (m / 16 + 64) * 2.0 ** -23) + 2.0 ** -21) * size + vanish + 2.0 ** -25 * (dtype == "f16")
    assert_within(out, ref, bound, "out")


@pytest.mark.parametrize("group", [1, 6, 12, 40])
@pytest.mark.parametrize("zeros", [slice(0, 200), slice(100, 300), slice(0, 300), slice(37, 38)])
def test_rows_of_zeros(zeros, group):
    """Histories that begin with, end with or are zero rows, as a padded prompt leaves them: scales, block scales and codes 0."""
    import torch
    c = Cache4([300, 5], 2, 64, 16, "bf16", seed=group)
    j = torch.arange(300, device="cuda")[zeros]
    for p in (c.k, c.v):
        p.put((c.table[0].long()[j // 16], slice(None), j % 16), torch.zeros((j.numel(), 2, 64), dtype=torch.uint8, device="cuda"), 0, 0.0)
    check(c, 2 * group)


def test_a_row_with_an_infinity_reads_as_no_number():
    import torch
    c = Cache4([40, 40], 1, 64, 8, "bf16", seed=3)
    c.v.scale[int(c.table[0, 2]), 0, 5] = math.inf
    c.v.block[int(c.table[0, 2]), 0, 5] = 0
    q, out, _, st = attend(c, 2)
    assert st == 0 and bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("page,group,shared", [(8, 2, False), (8, 12, True), (16, 33, False), (256, 2, False), (256, 8, True)])
def test_bad_pages_and_lengths_are_reported_and_spare_the_others(page, group, shared, dim):
    """Ids outside the pool at every place of a tile, in one box of many and in pages longer than a tile; lengths out of range."""
    import torch
    c = Cache4([900, 901, 40, 9], 2, dim, page, "bf16", shared=shared, seed=15)
    q, good, _, st = attend(c, 2 * group)
    assert st == 0
    ref, _, bound, _ = c.reference(q, dim ** -0.5)
    last = -(-900 // page) - 1
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        for e in sorted({0, 1, last // 2, last}):
            table = c.table.clone()
            c.table[0, e] = bad
            _, out, lse, st = attend(c, 2 * group)
            assert st == 3 and torch.equal(out[1:], good[1:])
            c.table.copy_(table)
    for bad in (-1, -2 ** 31, c.max_pages * page + 1, 2 ** 31 - 1):  # (another length, another split of the work: the others within their bounds)
        c.lens[3] = bad
        _, out, _, st = attend(c, 2 * group)
        assert st in (3, 6)
        assert_within(out[:3], ref[:3], bound[:3], "out")
        if bad < 0:
            assert st == 6 and not bool(out[3].any())
    c.lens[3] = 9
    _, out, _, st = attend(c, 2 * group)
    assert st == 0 and torch.equal(out, good)


# ---- append ----
def append(x, dim, page, layout="page", dtype="bf16", shared=True):
    """Rows x [n, heads, dim] into shuffled slots of a pool; returns the pool, the slots and a copy of what it held before."""
    import torch
    import cvr_ranking_model_gb300 as cvr
    from kv_util import cvr_type
    n, heads, _ = x.shape
    n_pages = -(-n // page) + 2
    p = Pool4(n_pages, heads, page, dim, layout)
    p.codes.fill_(0x5a)
    p.record.fill_(0xc3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:n].contiguous()
    cfg = cvr.make_kv_config(heads, heads, dim, page, n_pages, 1, 1, cvr_type(dtype), cvr.DTYPE_FP4, 0, p.codes.data_ptr(), p.strides(), p.record.data_ptr())
    kv = cvr.KvCache(cfg)
    kv.append(n, slots.data_ptr(), x.data_ptr(), k_stride=x.stride(0))
    kv.sync()
    return p, slots, kv


def check_rows(x, dim, page, **kw):
    import torch
    p, slots, kv = append(x, dim, page, **kw)
    code, block, scale = quantised(x)
    at = (slots // page, slice(None), slots % page)
    assert torch.equal(p.scale[at], scale)
    assert torch.equal(p.block[at], block)
    got = p.unpacked(*at)
    assert torch.equal(got & 7, code & 7)
    assert torch.equal((got >> 3)[(got & 7) > 0], (code >> 3)[(got & 7) > 0])  # (a zero may have either sign)
    rest = torch.ones(p.codes.shape[:1] + (page,), dtype=torch.bool, device="cuda")
    rest[slots // page, slots % page] = False
    assert bool((p.codes.transpose(1, 2)[rest] == 0x5a).all()) and bool((p.block.transpose(1, 2)[rest] == 0xc3).all())
    assert bool((p.scale.view(torch.int32).transpose(1, 2)[rest] == torch.tensor(0xc3c3c3c3 - 2 ** 32, device="cuda")).all())
    return p, slots, kv


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,page,layout", [(32, 3, 8, "page"), (64, 2, 16, "token"), (128, 5, 32, "gaps"), (128, 1, 256, "page")])
@pytest.mark.parametrize("kind", ["normal", "coarse", "bits"])
def test_appended_rows_are_the_exact_quotients(dtype, dim, heads, page, layout, kind):
    """Normal values; values of few bits, whose quotients meet ties; every exponent that the type has."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(dim)
    t = torch_type(dtype)
    n = 1000
    if kind == "normal":
        x = torch.randn((n, heads, dim + 8), generator=gen, device="cuda").to(t)
    elif kind == "coarse":
        x = torch.randint(-21, 22, (n, heads, dim + 8), generator=gen, device="cuda").to(t) * 0.25
    else:
        bits = torch.randint(-2 ** 15, 2 ** 15, (n, heads, dim + 8), generator=gen, device="cuda").to(torch.int16)
        x = bits.view(t)
        x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
        narrow = torch.randint(0, 2, (n, 1, 1), generator=gen, device="cuda").bool()  # half of the rows within few exponents
        few = (bits & (-0x1c01 if dtype == "f16" else -0x3f81)).view(t)
        x = torch.where(narrow & torch.isfinite(few), few, x)
    x = x.reshape(n, heads * (dim + 8))[:, :heads * dim]
    check_rows(x.unflatten(1, (heads, dim)), dim, page, layout=layout, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_appended_rows_at_the_ends(dtype):
    """Zero rows and blocks, one value among zeros, the type's largest and smallest numbers, blocks far below the row's largest."""
    import torch
    t = torch_type(dtype)
    tiny = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    top = torch.finfo(t).max
    x = torch.zeros((12, 1, 64), dtype=torch.float64, device="cuda")
    x[1, 0, 5] = 1.0
    x[2, 0, :] = top
    x[3, 0, ::2] = -top
    x[4, 0, :] = tiny
    x[5, 0, :3] = torch.tensor([tiny, -2 * tiny, 3 * tiny], dtype=torch.float64, device="cuda")
    x[6, 0, 0], x[6, 0, 16:32], x[6, 0, 32:48] = 1.0, 2.0 ** -18, 2.0 ** -19
    x[7, 0, 0], x[7, 0, 16:32], x[7, 0, 32:48] = 1.0, 1.75 * 2.0 ** -19, 2.0 ** -20
    x[8, 0, 0], x[8, 0, 63] = top, tiny
    x[9, 0, 16:32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2, dtype=torch.float64, device="cuda")
    x[10, 0, :16] = -x[9, 0, 16:32] * 2.0 ** -10
    x[11, 0, 0], x[11, 0, 16:32] = 448.0, torch.arange(1, 17, dtype=torch.float64, device="cuda") / 16
    check_rows(x.to(t), 64, 8, dtype=dtype)


def test_rows_with_infinities_and_nan():
    import torch
    x = torch.ones((4, 2, 32), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[1, 1, 31], x[2, 0, 0] = math.inf, math.nan, -math.inf
    p, slots, kv = append(x, 32, 8)
    s = p.scale[slots // 8, :, slots % 8]
    bad = torch.tensor([[1, 0], [0, 1], [1, 0], [0, 0]], device="cuda").bool()
    assert bool((~torch.isfinite(s) == bad).all())
    assert bool((p.codes[slots // 8, :, slots % 8][bad] == 0).all()) and bool((p.block[slots // 8, :, slots % 8][bad] == 0).all())
    out = torch.zeros_like(x)
    kv.read(4, slots.data_ptr(), out.data_ptr())
    kv.sync()
    assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == 1).all())


def test_padding_and_bad_slots():
    import torch
    x = torch.randn((5, 2, 64), device="cuda").to(torch.float16)
    p = Pool4(3, 2, 8, 64, "page")
    p.codes.fill_(1)
    p.record.fill_(2)
    import cvr_ranking_model_gb300 as cvr
    kv = cvr.KvCache(cvr.make_kv_config(2, 2, 64, 8, 3, 1, 1, cvr.DTYPE_F16, cvr.DTYPE_FP4, 0, p.codes.data_ptr(), p.strides(), p.record.data_ptr()))
    slots = torch.tensor([7, -1, 24, -2 ** 62, 2 ** 62], device="cuda")
    kv.append(5, slots.data_ptr(), x.data_ptr())
    assert kv.sync(check=False) == 3
    code, block, scale = quantised(x[:1])
    assert torch.equal(p.scale[0, :, 7], scale[0]) and torch.equal(p.block[0, :, 7], block[0]) and torch.equal(p.unpacked(0, slice(None), 7) & 7, code[0] & 7)
    p.codes[0, :, 7], p.block[0, :, 7], p.scale[0, :, 7] = 1, 2, 0
    p.scale.view(torch.int32)[0, :, 7] = 0x02020202
    assert bool((p.codes == 1).all()) and bool((p.record == 2).all())


# ---- read ----
@pytest.mark.parametrize("form", ["same", "i8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,layout,shared", [(32, "page", True), (64, "gaps", False), (128, "token", False)])
def test_rows_read_back(form, dtype, dim, layout, shared):
    """Repeated and padding slots among them; k and v as columns of one array."""
    import torch
    c = Cache4([70, 5, 300], 3, dim, 16, dtype, cache=form, layout=layout, shared=shared, seed=dim)
    j = torch.cat([c.slots(r, torch.arange(n, device="cuda")) for r, n in enumerate(c.lens_list)])
    want = torch.cat([torch.stack([torch.stack(c.rows(r, h, 0, n), 1) for h in range(3)], 2) for r, n in enumerate(c.lens_list)])  # [n, 2, h, d]
    pick = torch.randint(0, j.numel(), (501,), generator=c.gen, device="cuda")
    slots = j[pick].clone()
    slots[::7] = -1 - slots[::7]
    out = torch.full((501, 6 * dim + 8), 7.0, dtype=torch_type(dtype), device="cuda")
    kv = c.handle(3)
    kv.read(501, slots.data_ptr(), out.data_ptr(), 0 if shared else out[:, 3 * dim:].data_ptr(), out.stride(0), out.stride(0))
    kv.sync()
    assert bool((out[::7] == 7).all()) and bool((out[:, 6 * dim:] == 7).all())
    there = slots >= 0
    for w in range(1 if shared else 2):
        got, ref = out[there][:, w * 3 * dim:(w + 1) * 3 * dim].unflatten(1, (3, dim)), want[pick[there], w]
        # one rounding in fp32, one to the type
        step0 = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
        bound = torch.zeros_like(ref) if form == "same" else ref.abs() * (EPS[dtype] + 2.0 ** -23) + step0 / 2
        assert_within(got, ref, bound, "kv"[w])
    if not shared:  # v alone
        only = torch.zeros((501, 3, dim), dtype=torch_type(dtype), device="cuda")
        kv.read(501, slots.data_ptr(), 0, only.data_ptr())
        kv.sync()
        assert torch.equal(only[there], out[there][:, 3 * dim:6 * dim].unflatten(1, (3, dim)))


def test_reading_slots_outside_the_pool():
    import torch
    c = Cache4([20], 2, 64, 8, "bf16", seed=1)
    slots = torch.tensor([c.n_pages * 8, int(c.slots(0, torch.tensor([19], device="cuda"))), 2 ** 62, -2 ** 62], device="cuda")
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kv = c.handle(2)
    kv.read(4, slots.data_ptr(), out.data_ptr())
    assert kv.sync(check=False) == 3
    assert bool((out[[0, 2, 3]] == 7).all())
    assert_within(out[1], torch.stack([c.rows(0, h, 19, 20)[0][0] for h in range(2)]), torch.full((2, 64), 0.1, dtype=torch.float64, device="cuda"), "row")


@pytest.mark.parametrize("n", [1, 70001])
def test_appended_rows_come_back(n):
    import torch
    x = torch.randn((n, 2, 64), device="cuda").to(torch.bfloat16)
    p, slots, kv = append(x, 64, 64)
    out = torch.zeros_like(x)
    kv.read(n, slots.data_ptr(), out.data_ptr())
    kv.sync()
    ref = value_of(*quantised(x))
    assert_within(out, ref, ref.abs() * (EPS["bf16"] + 2.0 ** -23), "rows")
    # what a format of 4 bits is good for: a value is off by at most half a step of 2 (between 4 and 6), the block's scale by 2^-4
    big = x.double().unflatten(2, (4, 16)).abs().amax(-1, keepdim=True)
    assert bool(((x.double() - ref).unflatten(2, (4, 16)).abs() <= big / 6 * (1 + 2.0 ** -4) * 1.01 + big * 2.0 ** -4).all())


def test_refusals_of_read():
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache4([20], 2, 64, 8, "bf16", seed=1)
    kv = c.handle(2)
    x = torch.zeros((8, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(8, dtype=torch.int64, device="cuda")
    k, v, sl = x[:, 0].data_ptr(), x[:, 1].data_ptr(), s.data_ptr()
    for args, status in [((-1, sl, k, v, 256, 256), 2), ((2 ** 31, sl, k, v, 256, 256), 2), ((4, 0, k, v, 256, 256), 1), ((4, sl, 0, 0, 256, 256), 1), ((4, sl, k + 2, v, 256, 256), 1),
                         ((4, sl, k, v + 8, 256, 256), 1), ((4, sl + 4, k, v, 256, 256), 1), ((4, sl, k, v, 120, 256), 1), ((4, sl, k, v, 252, 256), 1), ((4, sl, k, k, 256, 256), 1),
                         ((4, sl, k, k + 128, 256, 256), 1), ((4, sl, k, v, 256, 512), 1), ((4, sl, k, sl, 256, 256), 1), ((4, sl, k, v, 256, 2 ** 62), 1)]:
        with pytest.raises(cvr.CvrError) as e:
            kv.read(*args)
        assert e.value.status == status, args
    kv.read(8, sl, k, v, 256, 256)
    kv.read(0, 0, 0)
    kv.sync()
    shared = Cache4([20], 2, 64, 8, "bf16", shared=True, seed=1).handle(2)
    with pytest.raises(cvr.CvrError):
        shared.read(4, sl, k, v, 256, 256)
    none = cvr.KvCache(cvr.make_kv_config(2, 2, 64, 8, 3, 1, 1))
    for call in (lambda: none.read(1, sl, k), lambda: none.weigh(1, k, sl, sl, 1.0, k, v), lambda: none.evict(1, sl, 4, 2, sl, k, v, sl + 8)):
        with pytest.raises(cvr.CvrError) as e:
            call()
        assert e.value.status == 1
