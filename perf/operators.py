"""Cases of the paged history cache's operators (the cvr_kv_* calls of include/cvr.h) for measurement.

Three operators, as a serving loop runs them for every step of its requests:
  tables  block tables and slot maps from request lengths: fresh pages from a free list, a slot for every new token
  append  the new tokens' key and value rows into their slots, in 16 bits or as 8-bit integers with a scale per row
  attend  one new query token per request and head over that request's pages, split over the length and joined

`own = False` computes them in elementary torch operations; `own = True` calls the library.
"""
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _attend(name, n_req, max_len, kv_heads, group, dim, page, **kw):
    c = dict(name=name, op="attend", n_req=n_req, min_len=1, max_len=max_len, skew=2.0, kv_heads=kv_heads, group=group, dim=dim, page=page,
             dtype="bf16", cache="same", shared=False, layout="page", window=0)
    c.update(kw)
    return c


def _append(name, n_tok, kv_heads, dim, page, **kw):
    c = dict(name=name, op="append", n_tok=n_tok, kv_heads=kv_heads, group=4, dim=dim, page=page, run=1, dtype="bf16", cache="same", layout="page")
    c.update(kw)
    return c


def _tables(name, n_req, max_len, page, **kw):
    c = dict(name=name, op="tables", n_req=n_req, min_len=1, max_len=max_len, skew=2.0, page=page, step="decode")
    c.update(kw)
    return c


def listed():
    return [
        # one visit: a single user's 200 conversions on the ranking model's heads, keys and values the same states (latency)
        _attend("attend_visit", 1, 200, 4, 1, 32, 16, min_len=200, shared=True),
        # a padded batch of users with browsing histories of up to 2000 events, empty rows among them
        _attend("attend_histories", 512, 2000, 4, 1, 32, 16, min_len=0, skew=1.0, shared=True),
        # an ordinary batch of grouped heads, ragged lengths, pages of one block per head
        _attend("attend_batch", 64, 8191, 8, 4, 128, 16),
        # one very long context, which only the split over its length spreads over the GPU
        _attend("attend_long", 1, 131071, 8, 4, 128, 64, min_len=131071, dtype="f16"),
        # the same kind of batch on an 8-bit cache with a scale per row
        _attend("attend_int8", 32, 16383, 8, 8, 128, 32, cache="int8"),
        # one key head for all query heads, rows of all heads together in a slot, only the last 1000 tokens seen
        _attend("attend_window", 48, 5001, 1, 16, 64, 32, min_len=0, dtype="f16", layout="token", window=1000),
        # a decode step's rows: one token for each of 64 requests
        _append("append_step", 64, 8, 128, 16),
        # prompts or back-filled histories: long runs of consecutive slots
        _append("append_prefill", 16383, 8, 128, 16, run=511),
        # the same into an 8-bit cache
        _append("append_int8", 2047, 8, 128, 32, run=200, cache="int8", layout="token", dtype="f16"),
        # a decode step's tables: every request grew by a token, a few need a fresh page
        _tables("tables_step", 64, 8191, 16),
        # a whole batch laid out from nothing: every page and every slot
        _tables("tables_fill", 4095, 4001, 16, step="fill"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "tables"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "tables":
        n = _log(rng, 1, 4095)
        return {k: v for k, v in _tables("", n, _log(rng, 2, min(16000, 16_000_000 // n)), page, min_len=rng.choice([0, 1]), skew=rng.choice([1.0, 2.0, 4.0]),
                                         step=rng.choice(["decode", "fill"])).items() if k != "name"}
    dim, dtype, cache = rng.choice([32, 64, 128]), rng.choice(["bf16", "f16"]), rng.choice(["same", "same", "int8"])
    kv, layout = rng.choice([1, 2, 4, 5, 8]), rng.choice(["page", "token"])
    row = kv * dim
    if op == "append":
        n = _log(rng, 1, min(16383, 16_000_000 // row if cache == "same" else 2_000_000 // row))
        return {k: v for k, v in _append("", n, kv, dim, page, run=_log(rng, 1, max(1, min(n, 2000))), dtype=dtype, cache=cache, layout=layout).items() if k != "name"}
    n = _log(rng, 1, 512)
    most = 100_000_000 // row
    top = _log(rng, 1, min(131071, max(1, most // n)))
    shared = rng.random() < 0.25
    window = _log(rng, 1, top) if rng.random() < 0.25 else 0
    return {k: v for k, v in _attend("", n, top, kv, rng.choice([1, 2, 3, 4, 8, 16, 24]), dim, page, min_len=rng.choice([0, 1, top]), skew=rng.choice([1.0, 2.0, 4.0]),
                                     dtype=dtype, cache=cache, shared=shared, layout=layout, window=window).items() if k != "name"}


# ---- what a case's sizes are, from the case alone ----
def _lens(case):
    """The requests' lengths in rising order: the longest is max_len, `skew` > 1 makes long ones rare."""
    n, lo, hi = case["n_req"], case["min_len"], case["max_len"]
    return [lo + int(round((hi - lo) * ((i + 1) / n) ** case["skew"])) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "tables":
        lens, page = _lens(case), case["page"]
        fill = case["step"] == "fill"
        new = [x if fill else min(x, 1) for x in lens]
        fresh = sum(_ceil(x, page) - (0 if fill else _ceil(x - y, page)) for x, y in zip(lens, new))
        slots = sum(new)
        # lengths, new tokens and held pages in; free pages in; table entries, slots, page counts and the list's head out; held pages under a new slot
        return {"bytes": 16.0 * len(lens) + 8.0 * fresh + 8.0 * slots + 8 + (0 if fill else 4.0 * slots), "flops": 0.0}
    size = 1 if case["cache"] == "int8" else 2
    if case["op"] == "append":
        rows = 2.0 * case["n_tok"] * case["kv_heads"]
        b = rows * case["dim"] * (2 + size) + 8.0 * case["n_tok"] + (4.0 * rows if size == 1 else 0)
        # the 8-bit rows come back as the values they stand for
        return {"bytes": b + (rows * (case["dim"] * 5 + 4) if size == 1 else 0), "flops": 0.0}
    seen = [min(x, case["window"]) if case["window"] else x for x in _lens(case)]
    heads = case["kv_heads"] * case["group"]
    row = case["dim"] * size + (4 if size == 1 else 0)
    b = sum(seen) * case["kv_heads"] * row * (1 if case["shared"] else 2) + sum(_ceil(x, case["page"]) for x in seen) * 4.0
    b += case["n_req"] * (heads * (2 * 2 * case["dim"] + 4) + 4)
    return {"bytes": float(b), "flops": 4.0 * sum(seen) * heads * case["dim"]}


# ---- inputs ----
def _pool(case, n_pages, gen):
    """A pool [page, head, token, dim] in the case's layout, and its row scales [page, head, token] (8 bits) or None."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    shape = (n_pages, p, h, d) if case["layout"] == "token" else (n_pages, h, p, d)
    x = torch.randn(shape, generator=gen, device="cuda")
    scale = None
    if case["cache"] == "int8":
        x = (x * 40.0).round_().clamp_(-127, 127).to(torch.int8)
        scale = torch.rand((n_pages, h, p), generator=gen, device="cuda") * 0.03 + 0.01
    else:
        x = x.to(_TYPES[case["dtype"]])
    return (x.permute(0, 2, 1, 3) if case["layout"] == "token" else x), scale


def _handle(case, n_pages, max_req, max_pages, k, k_scale, v, v_scale):
    import cvr_ranking_model_gb300 as cvr
    dt = {"bf16": cvr.DTYPE_BF16, "f16": cvr.DTYPE_F16}[case.get("dtype", "bf16")]

    def ptr(t):
        return 0 if t is None else t.data_ptr()

    cfg = cvr.make_kv_config(q_heads=case.get("kv_heads", 1) * case.get("group", 1), kv_heads=case.get("kv_heads", 1), head_dim=case.get("dim", 32),
                             page_size=case["page"], n_pages=n_pages, max_req=max_req, max_pages=max_pages, dtype=dt,
                             cache_dtype=cvr.DTYPE_I8 if case.get("cache") == "int8" else dt, window=case.get("window", 0),
                             k=ptr(k), k_strides=() if k is None else k.stride()[:3], k_scale=ptr(k_scale),
                             v=ptr(v), v_strides=() if v is None else v.stride()[:3], v_scale=ptr(v_scale))
    return cvr.KvCache(cfg, torch.cuda.current_stream().cuda_stream)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    page, s = case["page"], dict(case=case)
    if case["op"] == "append":
        n, h, d = case["n_tok"], case["kv_heads"], case["dim"]
        runs = _ceil(n, case["run"])  # runs of consecutive tokens, each in pages of its own from an offset of its own
        per = _ceil(case["run"] + page - 1, page)
        n_pages = runs * per + 3
        pages = torch.randperm(n_pages, generator=gen, device="cuda")[:runs * per].view(runs, per)
        i = torch.arange(n, device="cuda")
        r = i // case["run"]
        at = i % case["run"] + torch.randint(0, page, (runs,), generator=gen, device="cuda")[r]
        s["slots"] = pages[r, at // page] * page + at % page
        s["k"], s["k_scale"] = _pool(case, n_pages, gen)
        s["v"], s["v_scale"] = _pool(case, n_pages, gen)
        # the new rows are columns of a fused projection: query heads, then key heads, then value heads
        qkv = torch.randn((n, (case["group"] + 2) * h * d), generator=gen, device="cuda").to(_TYPES[case["dtype"]])
        s["k_new"], s["v_new"] = qkv[:, case["group"] * h * d:(case["group"] + 1) * h * d], qkv[:, (case["group"] + 1) * h * d:]
        if own:
            s["kv"] = _handle(case, n_pages, 1, 1, s["k"], s["k_scale"], s["v"], s["v_scale"])
        return s
    n, lens = case["n_req"], _lens(case)
    max_pages = max(1, _ceil(case["max_len"], page))
    need = sum(_ceil(x, page) for x in lens)
    n_pages = need + need // 16 + 61
    perm = torch.randperm(n, generator=gen, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[perm].contiguous()
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    if case["op"] == "attend":
        count = (s["lens"].long() + page - 1) // page
        first, j = count.cumsum(0) - count, torch.arange(max_pages, device="cuda")
        at = (first[:, None] + j).clamp_(max=n_pages - 1)
        s["table"] = torch.where(j < count[:, None], order[at], -1).to(torch.int32)
        s["k"], s["k_scale"] = _pool(case, n_pages, gen)
        s["v"], s["v_scale"] = (None, None) if case["shared"] else _pool(case, n_pages, gen)
        heads = case["kv_heads"] * case["group"]
        s["q"] = (torch.randn((n, heads, case["dim"]), generator=gen, device="cuda") * 2.0).to(_TYPES[case["dtype"]])
        s["scale"] = case["dim"] ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, heads), dtype=torch.float32, device="cuda")
        if own:
            s["kv"] = _handle(case, n_pages, n, max_pages, s["k"], s["k_scale"], s["v"], s["v_scale"])
        return s
    lens = s["lens"].long()
    new = lens if case["step"] == "fill" else lens.clamp(max=1)
    held = (lens - new + page - 1) // page
    s["new"], s["held"] = new.to(torch.int32), held.to(torch.int32)
    s["n_slots"] = sum(_lens(case)) if case["step"] == "fill" else sum(min(x, 1) for x in _lens(case))
    # the held pages are the first of the shuffled pool, the free list the others; the list's first entries are in use
    first, j = held.cumsum(0) - held, torch.arange(max_pages, device="cuda")
    s["table"] = torch.where(j < held[:, None], order[(first[:, None] + j).clamp_(max=n_pages - 1)], -1).to(torch.int32)
    s["free"] = order
    s["head"] = held.sum().to(torch.int32).reshape(1)
    s["pages"], s["head_out"] = torch.empty_like(s["held"]), torch.empty_like(s["head"])
    s["slots"] = torch.empty((max(1, s["n_slots"]),), dtype=torch.int64, device="cuda")
    if own:
        s["kv"] = _handle(case, n_pages, n, max_pages, None, None, None, None)
    return s


# ---- one pass ----
def run(s):
    return {"attend": _run_attend, "append": _run_append, "tables": _run_tables}[s["case"]["op"]](s)


def _run_attend(s):
    if own:
        q, out = s["q"], s["out"]
        s["kv"].attend(q.shape[0], q.data_ptr(), s["lens"].data_ptr(), s["table"].data_ptr(), s["scale"], out.data_ptr(), lse=s["lse"].data_ptr())
        return {"out": out, "lse": s["lse"]}
    c = s["case"]
    n, h, d = c["n_req"], c["kv_heads"], c["dim"]
    at = s["table"].clamp(min=0).long()

    def rows(pool, scale):  # [request, head, token, dim]
        x = pool[at].to(torch.float32)
        if scale is not None:
            x = x * scale[at][..., None]
        return x.transpose(1, 2).reshape(n, h, -1, d)

    k = rows(s["k"], s["k_scale"])
    v = k if c["shared"] else rows(s["v"], s["v_scale"])
    j, lens = torch.arange(k.shape[2], device="cuda"), s["lens"].long()[:, None]
    seen = j < lens
    if c["window"]:
        seen = seen & (j >= lens - c["window"])
    seen = seen[:, None, None, :]
    x = torch.matmul(s["q"].to(torch.float32).view(n, h, -1, d), k.transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(x - safe)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v * seen.transpose(2, 3)) / torch.where(total == 0, 1.0, total)
    lse = safe + torch.log(total)
    return {"out": o.reshape(n, -1, d).to(s["q"].dtype), "lse": lse.reshape(n, -1)}


def _run_append(s):
    c = s["case"]
    if own:
        k, v = s["k_new"], s["v_new"]
        s["kv"].append(c["n_tok"], s["slots"].data_ptr(), k.data_ptr(), v.data_ptr(), k_stride=k.stride(0), v_stride=v.stride(0))
        if c["cache"] != "int8":
            return {"k": s["k"], "v": s["v"]}
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]

    def put(pool, scale, new):
        x = new.reshape(c["n_tok"], c["kv_heads"], c["dim"])
        if scale is None:
            pool[page, :, at] = x
            return
        x = x.to(torch.float32)
        big = x.abs().amax(-1)
        # 127 x is exact in 32 bits and the one rounding of the quotient keeps a half a half: the same codes as in 64 bits
        code = torch.round(x * 127.0 / torch.where(big == 0, 1.0, big)[..., None])
        pool[page, :, at] = code.to(torch.int8)
        scale[page, :, at] = big / torch.full((), 127.0, device="cuda")

    if not own:
        put(s["k"], s["k_scale"], s["k_new"])
        put(s["v"], s["v_scale"], s["v_new"])
    if c["cache"] != "int8":
        return {"k": s["k"], "v": s["v"]}
    return {x: s[x][page, :, at].to(torch.float32) * s[x + "_scale"][page, :, at][..., None] for x in ("k", "v")}


def _run_tables(s):
    c = s["case"]
    if own:
        s["kv"].tables(c["n_req"], s["lens"].data_ptr(), s["table"].data_ptr(), new_lens=s["new"].data_ptr(), held=s["held"].data_ptr(),
                       free_pages=s["free"].data_ptr(), n_free=s["free"].numel(), free_head=s["head"].data_ptr(), pages=s["pages"].data_ptr(),
                       free_head_out=s["head_out"].data_ptr(), slots=s["slots"].data_ptr(), n_slots=s["n_slots"])
        return {"table": s["table"], "pages": s["pages"], "head": s["head_out"], "slots": s["slots"][:s["n_slots"]]}
    page, lens, new, held = c["page"], s["lens"].long(), s["new"].long(), s["held"].long()
    need = torch.maximum((lens + page - 1) // page, held)
    fresh = need - held
    first, j = s["head"].long() + fresh.cumsum(0) - fresh, torch.arange(s["table"].shape[1], device="cuda")
    at = (first[:, None] + j - held[:, None]).clamp_(min=0, max=s["free"].numel() - 1)
    table = torch.where((j >= held[:, None]) & (j < need[:, None]), s["free"][at], s["table"])
    ends = new.cumsum(0)
    i = torch.arange(s["n_slots"], device="cuda")
    r = torch.searchsorted(ends, i, right=True)
    pos = (lens - ends)[r] + i
    slots = table[r, pos // page].long() * page + pos % page
    return {"table": table, "pages": need.to(torch.int32), "head": (s["head"].long() + fresh.sum()).to(torch.int32), "slots": slots}


# ---- the definition in 64 bits ----
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        res = {}
        for x in ("k", "v"):
            new = s[x + "_new"].double().unflatten(1, (case["kv_heads"], case["dim"]))
            if case["cache"] == "int8":
                big = new.abs().max(dim=2, keepdim=True).values
                res[x] = torch.round(new * 127.0 / big.clamp(min=1e-300)) * big / 127.0
            else:
                flat = s[x].double().transpose(1, 2).flatten(0, 1)  # [slot, head, dim]
                flat[s["slots"]] = new
                res[x] = flat.unflatten(0, (-1, case["page"])).transpose(1, 2)
        return res
    g, page = case["group"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        ids = s["table"][r, lo // page:_ceil(n, page)].long()
        off = lo // page * page
        for h in range(case["kv_heads"]):
            def rows(x):
                t = s[x][ids, h].double()
                if s[x + "_scale"] is not None:
                    t = t * s[x + "_scale"][ids, h].double()[..., None]
                return t.flatten(0, 1)[lo - off:n - off]
            k = rows("k")
            v = k if case["shared"] else rows("v")
            x = s["q"][r, h * g:(h + 1) * g].double() @ k.T * s["scale"]
            out[r, h * g:(h + 1) * g] = torch.softmax(x, dim=1) @ v
            lse[r, h * g:(h + 1) * g] = torch.logsumexp(x, dim=1)
    return {"out": out, "lse": lse}
