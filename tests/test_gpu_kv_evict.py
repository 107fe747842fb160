"""cvr_kv_evict against its definition: which tokens stay, where their rows, scales and weights go, what is given back to the
free list, and every other place as it was; refusals and device-side errors; the operators together as decode steps."""
import math

import pytest

from kv_more_util import Cache4, evict_reference
from kv_util import assert_within, torch_type

pytestmark = pytest.mark.gpu


def dev(x, kind="int32"):
    import torch
    return torch.tensor(x, dtype=getattr(torch, kind), device="cuda")


def check(c, limit, keep, first=0, last=0, weight=None, held=None, free=True, seed=1, status=0, lens=None):
    """One call; all pools, weights, the list, the table and every output compared bit by bit."""
    import torch
    n, page = len(c.lens_list), c.page
    lens = c.lens_list if lens is None else lens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if weight is None:
        weight = torch.exp(torch.randn((c.n_pages, c.heads, page), generator=gen, device="cuda") * 2)
        weight = torch.where(torch.rand(weight.shape, generator=gen, device="cuda") < 0.3, weight.round(), weight)  # (ties)
    kept, after = evict_reference(c, lens, limit, keep, first, last, weight, c.table, page)
    stored = c.stored()
    want = [t.clone() for t in stored] + [weight.clone()]
    for (r, h), k in kept.items():
        i = torch.arange(keep, device="cuda")
        src, dst = c.table[r].long()[k.long() // page], c.table[r].long()[i // page]
        for t, old in zip(want, [*stored, weight]):
            t[dst, h, i % page] = old[src, h, k.long() % page]
    need = [-(-x // page) for x in lens]
    have = held or need
    left = [min(have[r], -(-keep // page)) if lens[r] > limit and free else have[r] for r in range(n)]
    back = [int(c.table[r, e]) for r in range(n) for e in range(left[r], have[r])]
    head, n_free = sum(have) + 3, sum(have) + 20
    pages_list = torch.randint(0, 1000, (n_free,), generator=gen, device="cuda").to(torch.int32)
    want_list = pages_list.clone()
    if free and back:
        want_list[head - len(back):head] = dev(back)
    table = c.table.clone()
    kept_out = torch.full((n + 1, c.heads, keep), -7, dtype=torch.int32, device="cuda")
    lens_out, pages = torch.full((n + 1,), -7, dtype=torch.int32, device="cuda"), torch.full((n + 1,), -7, dtype=torch.int32, device="cuda")
    t_head, t_out = dev([head]), dev([-7])
    t_held = None if held is None else dev(held)
    kv = c.handle(c.heads)
    got_weight = weight.clone()
    free_args = dict(free_pages=pages_list.data_ptr(), n_free=n_free, free_head=t_head.data_ptr(), free_head_out=t_out.data_ptr()) if free else {}
    kv.evict(n, c.lens.data_ptr(), limit, keep, c.table.data_ptr(), got_weight.data_ptr(), kept_out.data_ptr(), lens_out.data_ptr(), first, last,
             0 if held is None else t_held.data_ptr(), pages.data_ptr(), **free_args)
    assert kv.sync(check=False) == status
    for r in range(n):
        for h in range(c.heads):
            if (r, h) in kept:
                assert torch.equal(kept_out[r, h], kept[r, h]), (r, h)
            else:
                assert bool((kept_out[r, h] == -7).all()), (r, h)
    assert bool((kept_out[n] == -7).all()) and int(lens_out[n]) == -7 and int(pages[n]) == -7
    assert lens_out[:n].tolist() == after and pages[:n].tolist() == left
    assert torch.equal(table, c.table) and int(t_head) == head
    if free:
        assert int(t_out) == head - len(back) and torch.equal(pages_list, want_list)
    for t, w in zip([*stored, got_weight], want):
        kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
        assert torch.equal(t.view(kind), w.view(kind))
    return kv


@pytest.mark.parametrize("form", ["same", "i8", "fp4"])
@pytest.mark.parametrize("dim,heads,page,layout,shared", [(32, 4, 8, "page", True), (64, 3, 16, "gaps", False), (128, 2, 32, "token", False), (128, 1, 256, "page", False),
                                                          (32, 2, 64, "token", False), (64, 1, 8, "page", True), (128, 2, 16, "gaps", True)])
def test_forms_and_layouts(form, dim, heads, page, layout, shared):
    check(Cache4([0, 1, 99, 100, 101, 150, 400, 1001, 777], heads, dim, page, "bf16", cache=form, layout=layout, shared=shared, seed=dim), 100, 70, 3, 10)


@pytest.mark.parametrize("limit,keep,first,last", [(1, 1, 0, 0), (1, 1, 1, 0), (1, 1, 0, 1), (10, 10, 0, 0), (10, 10, 5, 5), (64, 17, 0, 17), (64, 17, 17, 0), (64, 17, 8, 9),
                                                   (64, 63, 1, 1), (500, 499, 0, 30), (513, 512, 0, 0), (1000, 1, 0, 0), (1000, 1000, 999, 0), (2000, 5, 1, 1)])
@pytest.mark.parametrize("form", ["same", "fp4"])
def test_limits(limit, keep, first, last, form):
    check(Cache4([0, 1, 2, 10, 11, 64, 65, 513, 514, 1000, 1001, 1500], 2, 64, 16, "f16", cache=form, seed=limit), limit, keep, first, last)


@pytest.mark.parametrize("n,limit,keep,first,last,heads,page", [(3000, 2500, 1200, 4, 100, 1, 16), (20000, 5000, 4097, 4, 128, 2, 64), (100000, 1, 1, 0, 0, 1, 256),
                                                                (100000, 90000, 80001, 100, 1000, 1, 16), (70001, 70000, 70000, 0, 0, 3, 8)])
def test_long_histories(n, limit, keep, first, last, heads, page):
    """One request, so that a cluster of CTAs shares a head, and shares longer than shared memory holds."""
    check(Cache4([n], heads, 32, page, "bf16", shared=True, seed=n), limit, keep, first, last)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "special", "bytes", "rising", "falling"])
@pytest.mark.parametrize("n", [300, 9000, 70000])
def test_weights_of_every_kind(kind, n):
    """All the same; few values; negative ones and both zeros; NaN and infinities; numbers that differ in one byte only; in order."""
    import torch
    c = Cache4([n], 1, 32, 32, "bf16", shared=True, seed=n)
    shape = (c.n_pages, 1, 32)
    gen = c.gen
    at = torch.argsort(c.table[0, :-(-n // 32)].long())  # (for order: a token's number from its page's place in the table)
    order = torch.zeros(shape, device="cuda")
    j = torch.arange(n, device="cuda")
    order[c.table[0].long()[j // 32], 0, j % 32] = j.float()
    assert at.numel() == -(-n // 32)
    w = {"equal": lambda: torch.full(shape, 0.25, device="cuda"),
         "few": lambda: torch.randint(0, 3, shape, generator=gen, device="cuda").float(),
         "signs": lambda: torch.randint(-2, 3, shape, generator=gen, device="cuda") * torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.5, 0.0, -1.0),
         "special": lambda: torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -math.nan], device="cuda")[
             torch.randint(0, 9, shape, generator=gen, device="cuda")],
         "bytes": lambda: (0x3f000000 + (torch.randint(0, 256, shape, generator=gen, device="cuda") << (8 * (n % 3)))).to(torch.int32).view(torch.float32),
         "rising": lambda: order, "falling": lambda: -order}[kind]()
    check(c, 250, 170, 3, 5, weight=w)
    check(c, 250, 170, 0, 0, weight=w)


def test_many_requests():
    """More requests than one CTA sums up, most of them not cut."""
    lens = [(i * 37) % 23 for i in range(1300)]
    check(Cache4(lens, 2, 32, 8, "bf16", seed=4), 20, 9, 1, 2)


def test_held_pages_and_no_list():
    """Requests that hold more pages than their tokens need give back those too; without a list nothing is given back."""
    c = Cache4([100, 30, 0, 64], 2, 64, 8, "bf16", seed=6)
    need = [13, 4, 0, 8]
    held = [n + x for n, x in zip(need, [2, 1, 2, 0])]
    check(c, 40, 20, held=held)
    check(Cache4([100, 30, 0, 64], 2, 64, 8, "bf16", seed=6), 40, 20, held=held, free=False)
    check(Cache4([100, 30, 0, 64], 2, 64, 8, "bf16", seed=6), 40, 20, free=False)


def test_no_request():
    import torch
    c = Cache4([10], 1, 32, 8, "bf16", seed=1)
    kv = c.handle(1)
    lst, head, out = torch.arange(5, dtype=torch.int32, device="cuda"), dev([3]), dev([-7])
    kv.evict(0, 0, 4, 2, 0, 0, 0, 0, free_pages=lst.data_ptr(), n_free=5, free_head=head.data_ptr(), free_head_out=out.data_ptr())
    kv.sync()
    assert int(out) == 3


def evict(c, kv, limit, keep, n_free=50, head=40, held=None, **kw):
    import torch
    n = len(c.lens_list)
    o = dict(weight=torch.rand((c.n_pages, c.heads, c.page), device="cuda"), kept=torch.zeros((n, c.heads, keep), dtype=torch.int32, device="cuda"),
             lens=torch.zeros(n, dtype=torch.int32, device="cuda"), pages=torch.zeros(n, dtype=torch.int32, device="cuda"),
             free=torch.full((n_free,), -5, dtype=torch.int32, device="cuda"), head=dev([head]), out=dev([-7]), held=None if held is None else dev(held))
    kv.evict(n, c.lens.data_ptr(), limit, keep, c.table.data_ptr(), o["weight"].data_ptr(), o["kept"].data_ptr(), o["lens"].data_ptr(),
             pages=o["pages"].data_ptr(), held=0 if held is None else o["held"].data_ptr(), free_pages=o["free"].data_ptr(), n_free=n_free,
             free_head=o["head"].data_ptr(), free_head_out=o["out"].data_ptr(), **kw)
    return o


def test_errors_on_the_device():
    import torch
    # no room in front of the list's head: the first pages are dropped, the others land
    c = Cache4([100, 90], 1, 64, 8, "bf16", seed=2)
    back = [int(c.table[r, e]) for r, n in ((0, 13), (1, 12)) for e in range(3, n)]
    kv = c.handle(1)
    o = evict(c, kv, 40, 20, head=7)
    assert kv.sync(check=False) == 8 and int(o["out"]) == 0 and o["free"].tolist() == back[-7:] + [-5] * 43
    # a list head out of range, used clamped
    for head, st in ((51, 6), (-1, 6)):
        c = Cache4([100], 1, 64, 8, "bf16", seed=2)
        kv = c.handle(1)
        o = evict(c, kv, 40, 20, head=head)
        assert kv.sync(check=False) == st and int(o["out"]) == (40 if head > 0 else 0)
    # lengths and held counts
    c = Cache4([100, 90], 1, 64, 8, "bf16", seed=2, max_pages=14)
    c.table[0, 13] = c.table[0, 0]
    c.lens[0], c.lens[1] = 10 ** 9, -1
    kv = c.handle(1)
    o = evict(c, kv, 120, 20)
    assert kv.sync(check=False) == 6 and o["lens"].tolist() == [112, 0]
    c = Cache4([100, 90], 1, 64, 8, "bf16", seed=2)
    kv = c.handle(1)
    o = evict(c, kv, 30, 20, held=[5, 12])
    assert kv.sync(check=False) == 6 and o["pages"].tolist() == [3, 3] and int(o["out"]) == 40 - 2 - 9 and o["lens"].tolist() == [20, 20]
    assert int(o["kept"][0].max()) < 40  # (of the tokens that the held pages have places for)
    o = evict(c, kv, 60, 20, held=[5, -1])
    assert kv.sync(check=False) == 6 and o["pages"].tolist() == [5, 0] and int(o["out"]) == 40 and o["lens"].tolist() == [40, 0]
    # a page outside the pool: reported, nothing out of the pools touched
    c = Cache4([100, 90], 1, 64, 8, "bf16", cache="same", seed=2)
    c.table[0, 1] = c.n_pages
    c.table[0, 5] = -1
    kv = c.handle(1)
    before = c.k.clone()
    o = evict(c, kv, 40, 20)
    assert kv.sync(check=False) == 3 and o["lens"].tolist() == [20, 20]
    others = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    others[c.table[0, [0, 2]].long()] = False
    others[c.table[1, :3].long()] = False
    assert torch.equal(c.k[others].view(torch.int16), before[others].view(torch.int16))
    kv.close()


def test_refusals():
    import torch
    import cvr_ranking_model_gb300 as cvr
    c = Cache4([20], 2, 64, 8, "bf16", seed=1)
    kv = c.handle(4)
    buf = torch.zeros(100000, dtype=torch.int32, device="cuda")
    lens, table, w, kept, out, held, pages, free, head, head_out = (buf[i * 5000:].data_ptr() for i in range(10))
    names = ["n", "lens", "limit", "keep", "table", "w", "kept", "out", "first", "last", "held", "pages", "free", "n_free", "head", "head_out"]
    ok = dict(zip(names, [1, lens, 10, 5, table, w, kept, out, 1, 2, held, pages, free, 100, head, head_out]))
    for change, status in [(dict(n=-1), 2), (dict(n=2), 2), (dict(limit=4), 2), (dict(keep=0), 2), (dict(keep=11), 2), (dict(limit=2 ** 30 + 1), 2), (dict(first=-1), 2), (dict(last=-1), 2),
                           (dict(first=4), 2), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), 2), (dict(n_free=-1), 2), (dict(n_free=2 ** 31 - 1), 2), (dict(free=0), 1), (dict(n_free=0), 1),
                           (dict(head=0), 1), (dict(head_out=0), 1), (dict(free=0, n_free=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(w=0), 1), (dict(kept=0), 1), (dict(out=0), 1),
                           (dict(out=lens), 1), (dict(pages=held), 1), (dict(pages=out), 1), (dict(head_out=head), 1), (dict(kept=table), 1), (dict(free=table), 1), (dict(w=kept), 1),
                           (dict(head_out=free + 396), 1)] + [({k: ok[k] + 2}, 1) for k in ("lens", "table", "w", "kept", "out", "held", "pages", "free", "head", "head_out")]:
        with pytest.raises(cvr.CvrError) as e:
            kv.evict(*{**ok, **change}.values())
        assert e.value.status == status, change


@pytest.mark.parametrize("form,dtype,dim,shared", [("same", "bf16", 64, False), ("fp4", "bf16", 128, False), ("i8", "f16", 32, True), ("fp4", "f16", 32, True)])
def test_decode_steps_of_all_operators(form, dtype, dim, shared):
    """Steps of tables, append, attend, weigh and evict over a cache that never grows beyond its limit, without waits, with waits and
    replayed from one captured graph: the same bits; the last step's attention against 64 bits on what the cache then holds."""
    import torch
    n, heads, group, page, limit, keep, steps = 5, 2, 3, 8, 40, 24, 90
    results = []
    for mode in ("eager", "waits", "graph"):
        c = Cache4([0] * n, heads, dim, page, dtype, cache=form, shared=shared, max_pages=8, spare=n * 6, seed=5)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(11)
        t = torch_type(dtype)
        rows = torch.randn((steps, 2, n, heads, dim), generator=gen, device="cuda").to(t)
        qs = torch.randn((steps, n, heads * group, dim), generator=gen, device="cuda").to(t)
        start = dev([0, 3, 9, 17, 39])
        start_pages = (start + page - 1) // page
        free = torch.randperm(c.n_pages, generator=gen, device="cuda").to(torch.int32)
        # the first histories: their tokens have slots, rows and a weight of zero
        pre = int(start.sum())
        slots0 = torch.zeros(pre, dtype=torch.int64, device="cuda")
        rows0 = torch.randn((2, pre, heads, dim), generator=gen, device="cuda").to(t)
        head, head2, held, held2 = dev([0]), dev([0]), torch.zeros_like(start), torch.zeros_like(start)
        weight = torch.zeros((c.n_pages, heads, page), device="cuda")
        c.table.fill_(-1)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        kv = c.handle(heads * group, stream=stream.cuda_stream)
        x = dict(lens=start.clone(), next=start.clone(), slots=torch.zeros(n, dtype=torch.int64, device="cuda"), k=torch.zeros_like(rows[0, 0]), v=torch.zeros_like(rows[0, 0]),
                 q=torch.zeros_like(qs[0]), out=torch.zeros_like(qs[0]), lse=torch.zeros((n, heads * group), device="cuda"),
                 kept=torch.zeros((n, heads, keep), dtype=torch.int32, device="cuda"))

        def first():
            kv.tables(n, start.data_ptr(), c.table.data_ptr(), start.data_ptr(), 0, free.data_ptr(), c.n_pages, head.data_ptr(), held2.data_ptr(), head2.data_ptr(),
                      slots0.data_ptr(), pre)
            kv.append(pre, slots0.data_ptr(), rows0[0].data_ptr(), 0 if shared else rows0[1].data_ptr())

        def step():
            x["lens"].copy_(x["next"] + 1)
            held.copy_(held2)
            head.copy_(head2)
            kv.tables(n, x["lens"].data_ptr(), c.table.data_ptr(), 0, held.data_ptr(), free.data_ptr(), c.n_pages, head.data_ptr(), held2.data_ptr(), head2.data_ptr(),
                      x["slots"].data_ptr(), n)
            wait()
            kv.append(n, x["slots"].data_ptr(), x["k"].data_ptr(), 0 if shared else x["v"].data_ptr())
            wait()
            kv.attend(n, x["q"].data_ptr(), x["lens"].data_ptr(), c.table.data_ptr(), dim ** -0.5, x["out"].data_ptr(), x["lse"].data_ptr())
            wait()
            kv.weigh(n, x["q"].data_ptr(), x["lens"].data_ptr(), c.table.data_ptr(), dim ** -0.5, x["lse"].data_ptr(), weight.data_ptr(), decay=0.95)
            wait()
            held.copy_(held2)
            head.copy_(head2)
            kv.evict(n, x["lens"].data_ptr(), limit, keep, c.table.data_ptr(), weight.data_ptr(), x["kept"].data_ptr(), x["next"].data_ptr(), 2, 8, held.data_ptr(), held2.data_ptr(),
                     free.data_ptr(), c.n_pages, head.data_ptr(), head2.data_ptr())
            wait()

        def wait():
            if mode == "waits":
                kv.sync()

        def feed(s):
            x["k"].copy_(rows[s, 0])
            x["v"].copy_(rows[s, 1])
            x["q"].copy_(qs[s])

        graph = torch.cuda.CUDAGraph()
        if mode == "graph":
            with torch.cuda.graph(graph, stream=stream):
                step()
            x["next"].copy_(start)
        torch.cuda.synchronize()
        trace = []
        with torch.cuda.stream(stream):
            first()
            for s in range(steps):
                feed(s)
                if mode == "graph":
                    graph.replay()
                else:
                    step()
                trace += [x["out"].clone(), x["kept"].clone(), x["next"].clone()]
        kv.sync()
        torch.cuda.synchronize()
        assert int(x["lens"].max()) <= limit + 1 and int(head2) == int(held2.sum())
        assert sorted(free[int(head2):].tolist() + [int(c.table[r, e]) for r in range(n) for e in range(int(held2[r]))]) == list(range(c.n_pages))
        results.append(trace + [weight.nan_to_num(), held2.clone(), free.clone()])
        c.lens_list = x["lens"].tolist()
        if mode == "eager" and all(m <= limit for m in c.lens_list):
            ref, _, bound, _ = c.reference(x["q"], dim ** -0.5)
            assert_within(x["out"], ref, bound, "out")
        assert any(bool((k >= keep).any()) for k in trace[1::3])  # (something was cut, later tokens among what stayed)
        kv.close()
        del start_pages
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("n_req,n", [(3, 100), (600, 100), (3, 5000), (400, 2500)])
def test_ids_outside_the_pool_are_not_given_back(n_req, n, heads):
    """Of the pages that cut requests no longer need those that are none of the pool are reported; the others close up to the list's head."""
    import torch
    lens = [n if r % 200 in (0, 1, 33) else 15 for r in range(n_req)]
    c = Cache4(lens, heads, 64, 8, "bf16", cache="same", seed=2)
    need = -(-n // 8)
    for r, e, bad in ((0, 5, -1), (0, need - 1, c.n_pages), (1, 3, 2 ** 31 - 1), (1, need // 2, c.n_pages + 7), (n_req - 1 - (n_req - 1) % 200, 4, -2 ** 31)):
        c.table[r, e] = bad
    ids = [i for r in range(n_req) if lens[r] == n for i in c.table[r, 3:need].tolist()]
    back = [i for i in ids if 0 <= i < c.n_pages]
    assert len(back) == len(ids) - 5
    kv, n_free = c.handle(heads), len(back) + 100
    for head in (len(back) + 50, len(back), len(back) - 3):
        o = evict(c, kv, 40, 20, n_free=n_free, head=head)
        assert kv.sync(check=False) == (3 if head >= len(back) else 8)
        there = back[max(0, len(back) - head):]
        begin = max(0, head - len(back))
        assert int(o["out"]) == begin and o["free"].tolist() == [-5] * begin + there + [-5] * (n_free - begin - len(there))
        assert o["lens"].tolist() == [20 if x == n else x for x in lens] and o["pages"].tolist() == [3 if x == n else 2 for x in lens]
    kv.close()


SHARED_OUT = [  # lens, heads, dim, page, layout, shared, limit, keep: what a (request, head) is cut by
    ([9000, 5, 4001], 2, 128, 16, "page", False, 2000, 1501),     # 8 CTAs of 256 threads
    ([5000, 4999, 300], 3, 64, 8, "gaps", False, 1000, 777),      # 4 of 256
    ([20000, 300], 2, 128, 32, "token", False, 12000, 9001),      # 8 of 1024
    ([33000, 16500], 2, 32, 64, "page", True, 3000, 2999),        # 8 of 1024
    ([18000, 2, 16400], 11, 32, 8, "page", False, 4000, 3333),    # 4 of 1024
    ([17000] + [300] * 99, 1, 64, 16, "page", False, 250, 129),   # one of 1024
]


@pytest.mark.parametrize("form", ["same", "i8", "fp4"])
@pytest.mark.parametrize("lens,heads,dim,page,layout,shared,limit,keep", SHARED_OUT)
def test_clusters_and_large_ctas(lens, heads, dim, page, layout, shared, limit, keep, form):
    """Rows of every size with their scales, one pool and two, moved by clusters and by CTAs of 1024 threads, over many rounds."""
    check(Cache4(lens, heads, dim, page, "bf16", cache=form, layout=layout, shared=shared, seed=len(lens) + dim), limit, keep, 3, 40)


@pytest.mark.parametrize("form", ["same", "fp4"])
@pytest.mark.parametrize("max_pages", [64, 256, 4096])
@pytest.mark.parametrize("limit,keep,first,last", [(1, 1, 0, 0), (4, 3, 1, 1), (300, 200, 0, 20)])
def test_short_histories_in_wide_tables(limit, keep, first, last, max_pages, form):
    """A table with room for far more tokens than there are: clusters most of whose CTAs have few tokens of a request or none."""
    check(Cache4([2, 3, 5, 0, 1, 40, 700], 2, 64, 16, "bf16", cache=form, max_pages=max_pages, seed=limit), limit, keep, first, last)


@pytest.mark.parametrize("form,dtype,dim,shared", [("same", "bf16", 64, False), ("i8", "f16", 32, True), ("fp4", "bf16", 128, False), ("fp4", "f16", 32, True)])
def test_attention_of_what_stays(form, dtype, dim, shared):
    """Steps of append, attend, weigh and evict, then the attention of the cut histories against 64 bits on what the cache holds."""
    import torch
    n, heads, group, page, limit, keep = 4, 2, 3, 8, 60, 33
    c = Cache4([60, 59, 40, 17], heads, dim, page, dtype, cache=form, shared=shared, max_pages=9, spare=30, seed=dim)
    for r in range(n):  # pages of its own for a request's next tokens
        have = -(-c.lens_list[r] // page)
        spare = sorted(set(range(c.n_pages)) - set(c.table[s, e].item() for s in range(n) for e in range(9 if s < r else -(-c.lens_list[s] // page))))
        c.table[r, have:] = dev(spare[:c.max_pages - have])
    assert len(set(c.table.flatten().tolist())) == n * c.max_pages
    kv, t = c.handle(heads * group), torch_type(dtype)
    weight, lens = torch.zeros((c.n_pages, heads, page), device="cuda"), list(c.lens_list)
    cuts, scale = 0, dim ** -0.5
    out, lse = torch.zeros((n, heads * group, dim), dtype=t, device="cuda"), torch.zeros((n, heads * group), device="cuda")
    kept, after = torch.zeros((n, heads, keep), dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    for _ in range(35):
        slots = torch.cat([c.slots(r, torch.tensor([lens[r]], device="cuda")) for r in range(n)])
        k, v = (torch.randn((n, heads, dim), generator=c.gen, device="cuda").to(t) for _ in range(2))
        q = torch.randn((n, heads * group, dim), generator=c.gen, device="cuda").to(t)
        c.lens.copy_(dev([x + 1 for x in lens]))
        kv.append(n, slots.data_ptr(), k.data_ptr(), 0 if shared else v.data_ptr())
        kv.attend(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, out.data_ptr(), lse.data_ptr())
        kv.weigh(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, lse.data_ptr(), weight.data_ptr())
        kv.evict(n, c.lens.data_ptr(), limit, keep, c.table.data_ptr(), weight.data_ptr(), kept.data_ptr(), after.data_ptr(), 2, 8)
        kv.sync()
        assert after.tolist() == [keep if x + 1 > limit else x + 1 for x in lens]
        cuts += sum(x + 1 > limit for x in lens)
        lens = after.tolist()
    assert cuts >= 5
    c.lens.copy_(after)
    c.lens_list = lens
    kv.attend(n, q.data_ptr(), c.lens.data_ptr(), c.table.data_ptr(), scale, out.data_ptr(), lse.data_ptr())
    kv.sync()
    ref, ref_lse, bound, b_lse = c.reference(q, scale)
    assert_within(out, ref, bound, "out")
    assert_within(lse, ref_lse, b_lse, "lse")
