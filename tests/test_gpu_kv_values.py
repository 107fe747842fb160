"""cvr_kv_attend at values where a range or a rounding inside the kernel could show. The bounds count the roundings that
include/cvr.h states."""
import math

import pytest

from kv_util import EPS, Cache, assert_within, torch_type

pytestmark = pytest.mark.gpu

GROUPS = [2, 12, 24, 40]  # one for each number of query rows that a tile is made for


def call(c, q, scale, window=0):
    import torch
    n, heads, _ = q.shape
    out, lse = torch.full_like(q, 7.0), torch.full((n, heads), 7.0, device="cuda")
    kv = c.handle(heads, window)
    kv.attend(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, out.data_ptr(), lse.data_ptr())
    kv.sync()
    return out, lse


def within(c, q, scale, out, split):
    """Against 64 bits, the bound free of what does not scale with the values. To first order:
      - logits: the D products' sum loses at most D 2^-23 of sum |q k| scale, the argument of the exponent 4 roundings of |s|;
        exp2 2^-21; both enter the numerator and the denominator, relative to sum p |v|;
      - the weights' split into two 16-bit halves: `split`, relative to sum p |v|;
      - sums over tokens: one add per 16 tokens and 64 for the joins, 2^-23 each, in numerator and denominator;
      - fp16 weights of 8-bit rows: per token 2^-33 of the row's largest weight times V scale, times codes of up to 127;
      - the output's rounding: half a step of it, or of the type's smallest subnormal."""
    import torch
    ref, bound = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    g, step0 = q.shape[1] // c.heads, {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}[c.dtype]
    for r in range(q.shape[0]):
        for h in range(c.heads):
            n = c.lens_list[r]
            k, v = c.rows(r, h, 0, n)
            j = torch.arange(n, device="cuda")
            v_scale = (c.k_scale if c.shared else c.v_scale)[c.table[r].long()[j // c.page], h, j % c.page].double().abs()
            rows = slice(h * g, (h + 1) * g)
            x = q[r, rows].double()
            s = x @ k.T * scale
            p = torch.softmax(s, 1)
            o, size = p @ v, p @ v.abs()
            ref[r, rows] = o
            logit = (x.abs() @ k.abs().T * abs(scale)).amax(1, keepdim=True) * c.dim * 2.0 ** -23 + s.abs().amax(1, keepdim=True) * 4 * 2.0 ** -24
            sums = (n / 16 + 64) * 2.0 ** -23
            vanish = 2.0 ** -33 * 127 * (p * v_scale).amax(1, keepdim=True) * n
            bound[r, rows] = EPS[c.dtype] * o.abs() + (2 * (logit + 2.0 ** -21 + sums) + split) * size + vanish + step0 / 2
    assert_within(out, ref, bound, "out")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("dim,shared", [(32, False), (64, False), (128, False), (64, True)])
@pytest.mark.parametrize("at", [[0], [2], [150, 299], [299]])
def test_a_large_value_without_weight_leaves_the_others_their_bits(dtype, group, dim, shared, at):
    """Tokens whose V scale is up to 2^40 times the others', which one half of the query rows gives a weight of about 2^-60 and
    the other half nearly all of its weight."""
    import torch
    n = 300
    c = Cache([n, 17], 2, dim, 16, dtype, "i8", shared=shared, seed=dim + group)
    q = torch.full((2, 2 * group, dim), 1.0, device="cuda")
    q[:, 1::2] = -1.0
    q += 0.01 * torch.randn(q.shape, generator=c.gen, device="cuda")
    q = q.to(torch_type(dtype))
    # (fp16: what the large ones give has to be in the type's range, and so do the others')
    small, large = {("bf16", False): (-6, 34), ("f16", False): (-19, 7), ("bf16", True): (-40, 0), ("f16", True): (-16, 0)}[dtype, shared]
    for r in range(2):
        p = c.table[r, :-(-c.lens_list[r] // 16)].long()
        c.k_scale[p] = 2.0 ** small if shared else 2.0 ** -13
        if not shared:
            c.v_scale[p] = 2.0 ** small
    for j in at:
        p, i = int(c.table[0, j // 16]), j % 16
        if shared:  # the logit and the value come from one row: -1 in every place
            c.k[p, :, i] = -1
            c.k_scale[p, :, i] = 1.0
        else:
            c.k[p, :, i] = -100
            c.k_scale[p, :, i] = 0.01
            c.v_scale[p, :, i] = 2.0 ** large
    scale = 42.0 / dim
    out, _ = call(c, q, scale)
    within(c, q, scale, out, 2.0 ** -21)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("log2_v", [-120, -108, -95, 90, 105])
def test_tiny_and_huge_row_scales_of_values(group, log2_v):
    import torch
    c = Cache([200, 3, 33], 2, 64, 16, "bf16", "i8", seed=group)
    c.v_scale *= 2.0 ** log2_v
    q = torch.randn((3, 2 * group, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
    out, _ = call(c, q, 0.125)
    within(c, q, 0.125, out, 2.0 ** -21)


def test_rising_and_falling_row_scales():
    """V scales that grow by 2^9 from tile to tile, or fall, under weights that fall or grow."""
    import torch
    for sign in (1, -1):
        c = Cache([640, 640], 1, 128, 64, "bf16", "i8", seed=5)
        q = torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda")
        q[:, 1] = -1
        for r in range(2):
            for j in range(10):
                p = int(c.table[r, j])
                c.v_scale[p] = 2.0 ** (sign * 9 * (j - 5))
                c.k[p] = 1 if r == 0 else -1
                c.k_scale[p] = 8.0 * j / 128
        out, _ = call(c, q, 1.0)
        within(c, q, 1.0, out, 2.0 ** -21)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("n,dim", [(700, 32), (20001, 128), (40000, 64)])
def test_scales_far_apart_in_histories_split_over_the_gpu(group, n, dim):
    """V scales from 2^-60 to 2^20 and zero ones, in any order."""
    import torch
    c = Cache([n, 5, 90], 1, dim, 64, "bf16", "i8", seed=n + group)
    e = torch.randint(-60, 21, c.v_scale.shape, generator=c.gen, device="cuda")
    c.v_scale *= torch.exp2(e.float())
    c.v_scale[torch.rand(c.v_scale.shape, generator=c.gen, device="cuda") < 0.2] = 0.0
    q = (torch.randn((3, group, dim), generator=c.gen, device="cuda") * 6).to(torch.bfloat16)
    out, lse = call(c, q, dim ** -0.5)
    within(c, q, dim ** -0.5, out, 2.0 ** -21)
    _, ref, _, bound = c.reference(q, dim ** -0.5)
    assert_within(lse, ref, bound, "lse")


@pytest.mark.parametrize("group", GROUPS)
def test_heavy_tokens_without_a_value(group):
    """Tokens that take nearly all the weight and whose value is zero: what the others leave keeps its bits."""
    import torch
    c = Cache([500, 40], 2, 64, 16, "f16", "i8", seed=group)
    for r in range(2):
        p = c.table[r, :-(-c.lens_list[r] // 16)].long()
        c.k_scale[p] = 2.0 ** -12
        for j in (0, 1, 37):
            c.k[int(c.table[r, j // 16]), :, j % 16] = 100
            c.k_scale[int(c.table[r, j // 16]), :, j % 16] = 0.01
            c.v_scale[int(c.table[r, j // 16]), :, j % 16] = 0.0
    q = torch.ones((2, 2 * group, 64), dtype=torch.float16, device="cuda")
    c.v_scale *= 2.0 ** 12
    out, _ = call(c, q, 18.0 / 64)
    within(c, q, 18.0 / 64, out, 2.0 ** -20)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_scale_that_is_no_number_among_scales_far_apart(group, bad):
    import torch
    c = Cache([300, 300], 1, 32, 16, "bf16", "i8", seed=group)
    c.v_scale *= torch.exp2(torch.randint(-30, 30, c.v_scale.shape, generator=c.gen, device="cuda").float())
    c.v_scale[int(c.table[0, 9]), 0, 3] = bad
    q = torch.randn((2, group, 32), generator=c.gen, device="cuda").to(torch.bfloat16)
    out, lse = call(c, q, 0.2)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("cache", ["same", "i8"])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("log2_q,log2_k,scale", [(70, 70, 2.0 ** -140), (70, 70, -2.0 ** -140), (100, 100, 0.0), (120, 90, 0.0), (-100, 100, 0.0),
                                                 (126, 60, 2.0 ** -140), (20, 100, 2.0 ** -120), (63, 63, 2.0 ** -126)])
def test_products_beyond_fp32_before_the_scale(cache, group, log2_q, log2_k, scale):
    """Only scale times q, the keys times 2^24 and the logits have to lie in fp32's range, not q . k."""
    import torch
    c = Cache([1, 50, 333], 2, 64, 16, "bf16", cache, seed=22)
    for r, n in enumerate(c.lens_list):
        p = c.table[r, :-(-n // 16)].long()
        if cache == "i8":
            c.k_scale[p] *= 2.0 ** log2_k
        else:
            c.k[p] = (c.k[p].float() * 2.0 ** log2_k).to(c.k.dtype)  # (exact: powers of two, far from the type's ends)
    q = (torch.randn((3, 2 * group, 64), generator=c.gen, device="cuda").clamp(-1.9, 1.9) * 2.0 ** log2_q).to(torch.bfloat16)
    out, lse = call(c, q, scale)
    ref, ref_lse, b_out, b_lse = c.reference(q, scale)
    assert_within(lse, ref_lse, b_lse, "lse")
    assert_within(out, ref, b_out, "out")


@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("log2", [10, 15, 16, 17, 40, 100, 127])
def test_one_huge_query_value_leaves_the_others_theirs(group, log2):
    """A query value that meets only zero keys: the logits are the other values', however much larger it is."""
    import torch
    c = Cache([3, 80], 2, 64, 16, "bf16", seed=log2)
    c.k[..., 11] = 0
    q = torch.randn((2, 2 * group, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
    small = q.clone()
    small[..., 11] = 0
    q[..., 11] = 2.0 ** log2
    out, lse = call(c, q, 0.125)
    ref, ref_lse, b_out, b_lse = c.reference(small, 0.125)
    assert_within(lse, ref_lse, b_lse, "lse")
    assert_within(out, ref, b_out, "out")


@pytest.mark.parametrize("cache", ["same", "i8"])
def test_a_scale_of_zero_keeps_what_is_no_number(cache):
    """0 times an infinity is no number: a scale of zero does not hide a bad query or key row, and spares the others."""
    import torch
    c = Cache([20, 20], 1, 32, 16, "bf16", cache, seed=3)
    q = torch.ones((2, 4, 32), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 3] = math.inf
    q[0, 2, 5] = math.nan
    if cache == "i8":
        c.k_scale[int(c.table[1, 0]), 0, 2] = math.inf
    else:
        c.k[int(c.table[1, 0]), 0, 2, 7] = math.inf
    out, lse = call(c, q, 0.0)
    assert bool(torch.isnan(out[0, 1:3]).all()) and bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    assert bool(torch.isfinite(out[0, [0, 3]]).all()) and bool(torch.isfinite(lse[0, [0, 3]]).all())


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "i8"), ("f16", "i8")])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("log2", [8, 14, 24, 31, 47, 100])
def test_logits_of_any_size_pick_the_largest(dtype, cache, group, apart, log2):
    """Logits are whole numbers times 2^log2, the largest of them once: its token's value is the output, its logit the lse."""
    import torch
    n = 120
    c = Cache([n], 2, 64, 16, dtype, cache, seed=log2)
    if cache == "i8":
        c.k_scale.fill_(1.0)
        if apart:  # (scales that give the rows bases of their own, less than 2^30 apart)
            c.v_scale *= torch.exp2(torch.randint(-20, 8, c.v_scale.shape, generator=c.gen, device="cuda").float())
    order = torch.randperm(n, generator=c.gen, device="cuda")
    for j in range(n):
        c.k[int(c.table[0, j // 16]), :, j % 16] = 0
        c.k[int(c.table[0, j // 16]), :, j % 16, 9] = int(order[j]) - 60
    q = torch.zeros((1, 2 * group, 64), dtype=torch_type(dtype), device="cuda")
    q[:, :, 9] = 8.0
    q[:, 1::2, 9] = -8.0
    out, lse = call(c, q, 2.0 ** (log2 - 3))
    for h in range(2):
        _, v = c.rows(0, h, 0, n)
        for i in range(group):
            best = int((order if i % 2 == 0 else -order).argmax())
            want, logit = v[best], float(order[best] - 60) * (1 if i % 2 == 0 else -1) * 2.0 ** log2
            # (the others weigh less than e^-250: their sum is below the output's smallest step. An output below its type's least
            # normal value rounds to half of the smallest subnormal, 2^-25 in fp16, where the far rows' values lie)
            bound = EPS[dtype] * want.abs() + 2.0 ** -20 * want.abs().amax() + {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}[dtype]
            assert bool(((out[0, h * group + i].double() - want).abs() <= bound).all())
            assert abs(float(lse[0, h * group + i]) - logit) <= abs(logit) * 2.0 ** -21


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "i8"), ("f16", "i8")])
@pytest.mark.parametrize("group", [1, 3, 16, 40])
def test_the_sum_of_few_weights_is_fp32(dtype, cache, group):
    """Two tokens, the first logit 0, the second s in (-0.7, 0): lse = ln(1 + e^s). Each logit is one exact product. What
    rounds: the exponent's factor and argument (3 half steps of |s| log2 e <= 1.01 at 2^-24, and with fp16 weights, whose
    exponents begin at 8, 2^-22) times ln 2, exp2 (2^-22 relative) and fp16's split (2^-22), all three times
    e^s / (1 + e^s) <= 1/2; the sum (2^-23 of it); ln and its scalings (4 half steps of 0.7). In all
    (3 * 2^-24 * 1.01 + 2^-22) ln 2 / 2 + 2^-23 + 2^-23 + 2^-23 + 0.7 * 4 * 2^-24 < 2^-20.5."""
    import torch
    n = 400
    c = Cache([2] * n, 1, 32, 8, dtype, cache, seed=group)
    p = c.table[:, 0].long()
    c.k[p, :, :2] = 0
    step = 64 if cache == "i8" else 1
    c.k[p, 0, 1, 5] = -step
    if cache == "i8":
        c.k_scale[p] = 1.0 / step
    q = torch.zeros((n, group, 32), device="cuda")
    q[:, :, 5] = torch.rand((n, group), generator=c.gen, device="cuda") * 0.69
    q = q.to(torch_type(dtype))
    _, lse = call(c, q, 1.0)
    want = torch.log1p(torch.exp(-q[:, :, 5].double()))
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -20.5


@pytest.mark.parametrize("dtype,cache,split", [("bf16", "same", 2.0 ** -16), ("f16", "same", 2.0 ** -22), ("bf16", "i8", 2.0 ** -22), ("f16", "i8", 2.0 ** -22)])
@pytest.mark.parametrize("group", GROUPS)
def test_weights_keep_both_halves(dtype, cache, split, group):
    """Eight tokens with exact logits in (-1, 0], values 1 and -1 in turn, so that the output is far below its sum p |v| = 1 and
    does not hide the weights' errors: the exponent's argument (2^-22 where exponents begin at 8, and 3 roundings of 2^-24) times
    ln 2 and exp2 (2^-22), below 2^-21 and twice, for numerator and denominator; the split; 8 adds of 2^-24, twice."""
    import torch
    n = 300
    c = Cache([8] * n, 1, 32, 8, dtype, cache, seed=group)
    p = c.table[:, 0].long()
    one = 64 if cache == "i8" else 1
    c.k[p] = 0
    c.k[p, 0, :, 5] = -torch.arange(1, 9, device="cuda").to(c.k.dtype) * (one // 8 if cache == "i8" else 0.125)
    c.v[p] = one
    c.v[p, 0, 1::2] = -one
    if cache == "i8":
        c.k_scale[p] = c.v_scale[p] = 1.0 / one
    q = torch.zeros((n, group, 32), device="cuda")
    q[:, :, 5] = torch.rand((n, group), generator=c.gen, device="cuda") * 0.02
    q = q.to(torch_type(dtype))
    out, _ = call(c, q, 1.0)
    s = -q[:, :, 5].double()[..., None] * torch.arange(1, 9, device="cuda") / 8
    w = torch.softmax(s, 2)
    want = (w[..., 0::2] - w[..., 1::2]).sum(2)[..., None]
    assert float(want.abs().max()) < 2.0 ** -8
    bound = EPS[dtype] * want.abs() + 2 * 2.0 ** -21 + split + 2 * 8 * 2.0 ** -24 + 2.0 ** -25
    assert bool(((out.double() - want).abs() <= bound).all())
