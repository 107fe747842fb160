"""cvr_kv_weigh against its definition in 64 bits: pool types, head layouts, lengths around a block's size, decay, new tokens,
places that must stay as they are; its refusals and device-side errors."""
import math

import pytest

from kv_more_util import Cache4
from kv_util import assert_within, torch_type

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513]
FORMS = ["same", "i8", "fp4"]


def exact_lse(c, q, scale):
    import torch
    n, heads, _ = q.shape
    g = heads // c.heads
    lse = torch.full((n, heads), -math.inf, device="cuda")
    for r in range(n):
        m = min(max(c.lens_list[r], 0), c.max_pages * c.page)
        for h in range(c.heads if m else 0):
            k, _ = c.rows(r, h, 0, m)
            lse[r, h * g:(h + 1) * g] = torch.logsumexp(q[r, h * g:(h + 1) * g].double() @ k.T * scale, 1).float()
    return lse


def check(c, q_heads, decay=1.0, new=None, scale=None, gain=1.0, lse=None, seed=3, status=0):
    import torch
    n = len(c.lens_list)
    scale = c.dim ** -0.5 if scale is None else scale
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    wide = torch.full((n, q_heads * c.dim + 8), math.nan, dtype=torch_type(c.dtype), device="cuda")
    wide[:, :q_heads * c.dim] = (torch.randn((n, q_heads * c.dim), generator=gen, device="cuda") * gain).to(wide.dtype)
    q = wide[:, :q_heads * c.dim].unflatten(1, (q_heads, c.dim))
    lse = exact_lse(c, q, scale) if lse is None else lse
    weight = torch.rand((c.n_pages, c.heads, c.page), generator=gen, device="cuda")
    counts = [min(1, max(0, x)) for x in c.lens_list] if new is None else new
    for r, m in enumerate(c.lens_list):  # what must not be read: weights of new tokens, or all of them
        j = torch.arange(max(0, min(m, c.max_pages * c.page) - counts[r]) if decay else 0, max(0, min(m, c.max_pages * c.page)), device="cuda")
        weight[c.table[r].long()[j // c.page], :, j % c.page] = math.nan
    got = weight.clone()
    kv = c.handle(q_heads)
    new_lens = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    kv.weigh(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, lse.data_ptr(), got.data_ptr(), decay, 0 if new is None else new_lens.data_ptr(),
             wide.stride(0))
    assert kv.sync(check=False) == status
    ref, bound = c.weigh_reference(q, scale, lse, weight, decay, counts)
    assert_within(got, ref, bound, "weight")
    return got, q, lse


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("heads,group", [(4, 1), (2, 4), (3, 8), (1, 12), (1, 17), (1, 64)])
def test_types_dims_and_heads(form, dtype, dim, heads, group):
    check(Cache4(EDGES, heads, dim, 16, dtype, cache=form, seed=dim + group), heads * group)


@pytest.mark.parametrize("layout", ["page", "token", "gaps"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim,form", [(32, "fp4"), (64, "i8"), (128, "same"), (128, "fp4")])
def test_pages_and_pool_layouts(layout, page, dim, form):
    check(Cache4([300, 0, 1, page - 1, page, page + 1, 777], 3, dim, page, "bf16", cache=form, layout=layout, seed=page), 6)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, 3.0])
@pytest.mark.parametrize("new", [None, "none", "some", "all"])
def test_decay_and_new_tokens(form, decay, new):
    lens = [0, 1, 5, 16, 33, 200]
    count = {None: None, "none": [0] * 6, "some": [0, 0, 3, 16, 1, 100], "all": lens}[new]
    check(Cache4(lens, 2, 64, 8, "f16", cache=form, seed=7), 6, decay, count)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,heads,group,dim", [(70001, 1, 1, 32), (20001, 8, 4, 128), (30000, 2, 24, 64)])
def test_long_histories(form, n, heads, group, dim):
    check(Cache4([n], heads, dim, 64, "bf16", cache=form, seed=n), heads * group)


def test_ragged_batch_long_and_short():
    check(Cache4([5000, 1, 0, 0, 64, 12345, 3, 700] + [0] * 40 + [9] * 30, 2, 128, 16, "f16", seed=3), 8)


def test_many_requests_most_of_them_empty():
    """More requests than a CTA has threads, so that a thread sums several; windows of 32 empty ones on the way."""
    lens = [3 if i % 97 == 0 else 40 if i == 2999 else 0 for i in range(3000)]
    check(Cache4(lens, 2, 32, 8, "bf16", seed=18), 2)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 40.0])
@pytest.mark.parametrize("form", FORMS)
def test_scales(scale, form):
    check(Cache4([1, 50, 333], 2, 64, 16, "bf16", cache=form, seed=8), 4, scale=scale)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("log2_q,log2_k,scale", [(126, -90, 2.0 ** -38), (-130, 100, 2.0 ** 28)])
def test_queries_at_the_ends_of_bf16(log2_q, log2_k, scale, form):
    c = Cache4([1, 50, 333], 2, 64, 16, "bf16", cache=form, seed=22)
    if form == "same":
        for r, n in enumerate(c.lens_list):
            p = c.table[r, :-(-n // 16)].long()
            c.k[p] = (c.k[p].float() * 2.0 ** log2_k).to(c.k.dtype)
    else:
        (c.k_scale if form == "i8" else c.k.scale).mul_(2.0 ** log2_k)
    check(c, 4, scale=scale, gain=0.9 * 2.0 ** log2_q)


def test_weights_of_the_attention_add_up_to_one_per_head():
    """lse from cvr_kv_attend, on the same queries: over a request's tokens the weights of a kv head sum to its query heads. Each is off by
    what weigh's bound says plus the lse's, about 1e-5 here."""
    import torch
    for form in FORMS:
        c = Cache4([1, 700, 33], 2, 64, 16, "bf16", cache=form, seed=4)
        q = torch.randn((3, 8, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
        out, lse, weight = torch.zeros_like(q), torch.zeros((3, 8), device="cuda"), torch.full((c.n_pages, 2, 16), math.nan, device="cuda")
        kv = c.handle(8)
        kv.attend(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.125, out.data_ptr(), lse.data_ptr())
        kv.weigh(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.125, lse.data_ptr(), weight.data_ptr(), decay=0.0)
        kv.sync()
        for r, n in enumerate(c.lens_list):
            j = torch.arange(n, device="cuda")
            total = weight[c.table[r].long()[j // 16], :, j % 16].double().sum(0)
            assert bool(((total - 4).abs() < 4e-5).all()), (form, r, total)


@pytest.mark.parametrize("group", [1, 3, 12, 20])
def test_keys_with_infinities(group):
    """A logit of -infinity weighs nothing, one of infinity infinitely much, whatever heads the products' tiles are filled up with."""
    import torch
    c = Cache4([40], 1, 64, 8, "bf16", cache="same", seed=1)
    q = torch.ones((1, group, 64), dtype=torch.bfloat16, device="cuda")
    c.k[int(c.table[0, 1]), 0, 3, 7], c.k[int(c.table[0, 2]), 0, 3, 7] = -math.inf, math.inf
    lse, weight = torch.zeros((1, group), device="cuda"), torch.zeros((c.n_pages, 1, 8), device="cuda")
    kv = c.handle(group)
    kv.weigh(1, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.01, lse.data_ptr(), weight.data_ptr(), decay=0.0)
    kv.sync()
    got = weight[c.table[0, :5].long(), 0].flatten()
    assert float(got[11]) == 0 and float(got[19]) == math.inf and bool(torch.isfinite(torch.cat([got[:19], got[20:]])).all())


def test_the_same_bits_on_every_call():
    import torch
    c = Cache4([5000, 3, 777], 2, 128, 16, "bf16", cache="fp4", seed=9)
    first = check(c, 24)[0]
    for _ in range(3):
        assert torch.equal(torch.nan_to_num(check(c, 24)[0]), torch.nan_to_num(first))


def test_bad_lengths_and_pages():
    """Lengths are clamped and reported; the tokens of a page outside the pool are left out."""
    import torch
    c = Cache4([20, -3, 40], 2, 64, 8, "bf16", seed=1, max_pages=5)
    c.lens[0] = 10 ** 6
    c.table[0, 3:5] = c.table[0, :2]  # (somewhere valid: the clamped length reads them)
    c.lens_list[0] = 40
    q = torch.randn((3, 4, 64), generator=c.gen, device="cuda").to(torch.bfloat16)
    kv, lse, weight = c.handle(4), torch.zeros((3, 4), device="cuda"), torch.zeros((c.n_pages, 2, 8), device="cuda")
    kv.weigh(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, lse.data_ptr(), weight.data_ptr())
    assert kv.sync(check=False) == 6
    c = Cache4([20, 17], 2, 64, 8, "bf16", seed=1)
    c.table[0, 1] = c.n_pages
    c.table[1, 2] = -1
    weight = torch.full((c.n_pages, 2, 8), 5.0, device="cuda")
    kv, zeros = c.handle(4), torch.zeros(2, dtype=torch.int32, device="cuda")
    kv.weigh(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, lse.data_ptr(), weight.data_ptr(), new_lens=zeros.data_ptr())
    assert kv.sync(check=False) == 3
    touched = (weight != 5).any(1)
    want = torch.zeros_like(touched)
    for r, tokens in ((0, [*range(8), *range(16, 20)]), (1, range(16))):
        j = torch.tensor(list(tokens), device="cuda")
        want[c.table[r].long()[j // 8], j % 8] = True
    assert torch.equal(touched, want)
    bad_new = torch.tensor([21, -1], dtype=torch.int32, device="cuda")
    c = Cache4([20, 17], 2, 64, 8, "bf16", seed=1)
    kv = c.handle(4)
    kv.weigh(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, lse.data_ptr(), weight.data_ptr(), new_lens=bad_new.data_ptr())
    assert kv.sync(check=False) == 6


def test_refusals():
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache4([20], 2, 64, 8, "bf16", seed=1)
    kv = c.handle(4)
    buf = torch.zeros(100000, device="cuda")
    q, lens, table, lse, w = (buf[i * 1000:].data_ptr() for i in (0, 1, 2, 3, 10))
    ok = (1, q, lens, table, 0.1, lse, w, 1.0, 0, 0)

    def changed(**kw):
        names = ["n", "q", "lens", "table", "scale", "lse", "w", "decay", "new", "stride"]
        return [kw.get(k, v) for k, v in zip(names, ok)]

    for change, status in [(dict(n=-1), 2), (dict(n=2), 2), (dict(q=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(lse=0), 1), (dict(w=0), 1), (dict(scale=math.inf), 1),
                           (dict(scale=math.nan), 1), (dict(decay=-0.5), 1), (dict(decay=math.inf), 1), (dict(decay=math.nan), 1), (dict(q=q + 8), 1), (dict(lens=lens + 2), 1),
                           (dict(w=w + 1), 1), (dict(lse=lse + 2), 1), (dict(new=lens + 1), 1), (dict(stride=252), 1), (dict(stride=248), 1), (dict(w=lse), 1), (dict(w=q), 1), (dict(w=lens), 1),
                           (dict(w=table), 1), (dict(new=w), 1)]:
        with pytest.raises(cvr.CvrError) as e:
            kv.weigh(*changed(**change))
        assert e.value.status == status, change
    kv.weigh(*changed(n=0, q=0))
    kv.sync()
    windowed = Cache4([20], 2, 64, 8, "bf16", seed=1).handle(4, window=5)
    with pytest.raises(cvr.CvrError) as e:
        windowed.weigh(*ok)
    assert e.value.status == 1
    with pytest.raises(cvr.CvrError) as e:
        windowed.evict(1, lens, 4, 2, table, w, lse, q)
    assert e.value.status == 1


def test_two_threads_with_handles_of_their_own():
    """Handles of different numbers of query heads, whose launches of one kernel ask for different amounts of shared memory, each on a stream
    and in a thread of its own: every call is taken, and the weights are those of a call alone."""
    import threading
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache4([40, 7], 1, 128, 16, "bf16", cache="same", seed=2)
    jobs = []
    for group in (24, 64):
        q = torch.randn((2, group, 128), generator=c.gen, device="cuda").to(torch.bfloat16)
        lse, stream = exact_lse(c, q, 0.1), torch.cuda.Stream()
        alone, got = (torch.zeros((c.n_pages, 1, 16), device="cuda") for _ in range(2))
        kv = c.handle(group)
        kv.weigh(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, lse.data_ptr(), alone.data_ptr(), decay=0.0)
        kv.sync()
        jobs.append((c.handle(group, stream=stream.cuda_stream), q, lse, alone, got, stream))
    torch.cuda.synchronize()
    refused, start = [], threading.Barrier(2)

    def work(kv, q, lse, alone, got, stream):
        start.wait()
        for _ in range(20000):
            try:
                kv.weigh(2, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 0.1, lse.data_ptr(), got.data_ptr(), decay=0.0)
            except cvr.CvrError as e:
                refused.append(str(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for kv, _, _, alone, got, _ in jobs:
        kv.sync()
        assert torch.equal(got, alone)
    assert not refused, (len(refused), refused[0])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [3, 12, 20])
@pytest.mark.parametrize("log2", [10, 20, 24, 31, 60])
def test_large_logits_weigh_at_most_one_per_head(log2, group, dtype, form):
    """Logits about 2^log2 and their lse are off by 2^-23 of themselves and more, and a weight by e to the power of that. With lse from the
    attention of the same queries no query head gives a token more than 1 for it (exp2 itself is off by at most 2^-21)."""
    import torch
    c = Cache4([1, 700, 33], 2, 64, 16, dtype, cache=form, seed=group)
    q = torch.randn((3, 2 * group, 64), generator=c.gen, device="cuda").to(torch_type(dtype))
    out, lse, weight = torch.zeros_like(q), torch.zeros((3, 2 * group), device="cuda"), torch.full((c.n_pages, 2, 16), math.nan, device="cuda")
    kv = c.handle(2 * group)
    kv.attend(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 2.0 ** (log2 - 3), out.data_ptr(), lse.data_ptr())
    kv.weigh(3, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), 2.0 ** (log2 - 3), lse.data_ptr(), weight.data_ptr(), decay=0.0)
    kv.sync()
    assert bool(torch.isfinite(lse).all())
    for r, n in enumerate(c.lens_list):
        j = torch.arange(n, device="cuda")
        w = weight[c.table[r].long()[j // 16], :, j % 16]
        assert bool((w >= 0).all()) and float(w.max()) <= group * (1 + 2.0 ** -21), (r, float(w.max()))
