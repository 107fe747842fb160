"""Cases of the operators that let a paged history cache hold more in the same memory, for measurement.

Five operators on the pools and block tables of the cvr_kv_* calls of include/cvr.h:
  append  new key and value rows into pools of 4 bits: e2m1 codes, an e4m3 scale per 16 values, an fp32 scale per row
  read    rows of given slots back as values of 16 bits
  attend  one new query token per request and head over pages of 4 bits
  weigh   what each cached token's attention weight of a query token adds up to, per key head
  evict   histories over a limit cut to their heaviest tokens, in place, their free pages back to the list

`own = False` computes them in elementary torch operations; `own = True` calls the library.
"""
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _rows(op, name, n_tok, kv_heads, dim, page, **kw):
    c = dict(name=name, op=op, n_tok=n_tok, kv_heads=kv_heads, group=4, dim=dim, page=page, run=1, dtype="bf16", cache="fp4", shared=False, layout="page")
    c.update(kw)
    return c


def _requests(op, name, n_req, max_len, kv_heads, group, dim, page, **kw):
    c = dict(name=name, op=op, n_req=n_req, min_len=1, max_len=max_len, skew=2.0, kv_heads=kv_heads, group=group, dim=dim, page=page, dtype="bf16",
             cache="fp4", shared=False, layout="page")
    if op == "weigh":
        c.update(cache="same", decay=1.0)
    if op == "evict":
        c.update(cache="same", keep=max(1, max_len // 8), limit=max(1, max_len // 4), first=0, last=0)
    c.update(kw)
    return c


def listed():
    return [
        # a decode step's rows: one token for each of 64 requests, rows of a fused projection
        _rows("append", "append_step", 64, 8, 128, 16),
        # prompts or back-filled histories: long runs of consecutive slots
        _rows("append", "append_prefill", 16383, 8, 128, 16, run=511),
        # one visit's history back in 16 bits, keys and values the same states (latency)
        _rows("read", "read_visit", 200, 4, 32, 16, run=200, dtype="f16", shared=True),
        # cached prefixes back in 16 bits, for a prompt's attention elsewhere
        _rows("read", "read_prefix", 16383, 8, 128, 32, run=2000, layout="token"),
        # one visit: a single user's 200 conversions on the ranking model's heads, keys and values the same states (latency)
        _requests("attend", "attend_visit", 1, 200, 4, 1, 32, 16, min_len=200, shared=True),
        # an ordinary batch of grouped heads, ragged lengths
        _requests("attend", "attend_batch", 64, 8191, 8, 4, 128, 16),
        # one very long context, which only a split over its length spreads over the GPU
        _requests("attend", "attend_long", 1, 131071, 8, 4, 128, 64, min_len=131071, dtype="f16"),
        # one key head for sixteen query heads, rows of all heads together in a slot, empty histories among them
        _requests("attend", "attend_groups", 48, 16001, 2, 16, 64, 32, min_len=0, dtype="f16", layout="token"),
        # a decode step's weights on the ordinary batch, summed over the whole life of the tokens
        _requests("weigh", "weigh_batch", 64, 8191, 8, 4, 128, 16),
        # the same for few, longer requests on 4 bits, old weights fading
        _requests("weigh", "weigh_fp4", 32, 16383, 8, 8, 128, 32, cache="fp4", decay=0.99),
        # browsing histories of the ranking model's heads cut to 256 events, the newest 32 of them untouched
        _requests("evict", "evict_histories", 16, 2000, 4, 1, 32, 16, min_len=0, skew=1.0, shared=True, limit=512, keep=256, last=32),
        # a batch of prompts cut to an eighth, its first tokens and the recent ones kept
        _requests("evict", "evict_batch", 64, 8191, 8, 4, 128, 16, skew=1.0, limit=2048, keep=1023, first=4, last=128),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "weigh", "weigh", "evict", "evict"])
    page, dim, dtype = rng.choice([8, 16, 32, 64, 128, 256]), rng.choice([32, 64, 128]), rng.choice(["bf16", "f16"])
    kv, layout, shared = rng.choice([1, 2, 4, 5, 8]), rng.choice(["page", "token"]), rng.random() < 0.25
    row = kv * dim
    same = dict(dtype=dtype, layout=layout, shared=shared)
    if op in ("append", "read"):
        n = _log(rng, 1, min(16383, 16_000_000 // row))
        c = _rows(op, "", n, kv, dim, page, run=_log(rng, 1, max(1, min(n, 2000))), cache="fp4" if op == "append" else rng.choice(["fp4", "int8", "same"]), **same)
    else:
        n = _log(rng, 1, 512 if op != "evict" else 96)
        most = (100_000_000 if op != "evict" else 60_000_000) // row
        top = _log(rng, 1 if op != "evict" else 8, min(131071, max(8, most // n)))
        kw = dict(min_len=rng.choice([0, 1, top]), skew=rng.choice([1.0, 2.0, 4.0]), **same)
        if op == "weigh":
            kw.update(cache=rng.choice(["same", "int8", "fp4"]), decay=rng.choice([1.0, 0.9, 0.0]))
        if op == "evict":
            limit = _log(rng, 2, max(2, top - 1))
            keep = _log(rng, 1, limit)
            last = rng.choice([0, keep // 8, keep // 2])
            kw.update(cache=rng.choice(["same", "same", "int8", "fp4"]), limit=limit, keep=keep, last=last, first=rng.choice([0, min(4, keep - last)]))
        c = _requests(op, "", n, top, kv, rng.choice([1, 2, 3, 4, 8, 16, 24]), dim, page, **kw)
    return {k: v for k, v in c.items() if k != "name"}


# ---- what a case's sizes are, from the case alone ----
def _lens(case):
    """The requests' lengths in rising order: the longest is max_len, `skew` > 1 makes long ones rare."""
    n, lo, hi = case["n_req"], case["min_len"], case["max_len"]
    return [lo + int(round((hi - lo) * ((i + 1) / n) ** case["skew"])) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _row_bytes(case):
    """A row as the pool holds it, its scales included."""
    d = case["dim"]
    return {"same": 2 * d, "int8": d + 4, "fp4": d // 2 + d // 16 + 4}[case["cache"]]


def work(case):
    h, d, pools, row = case["kv_heads"], case["dim"], 1 if case["shared"] else 2, _row_bytes(case)
    if case["op"] in ("append", "read"):
        rows = pools * case["n_tok"] * h
        # appended rows come back as the values they stand for: both directions
        return {"bytes": float(rows * (2 * d + row) * (2 if case["op"] == "append" else 1) + 8 * case["n_tok"]), "flops": 0.0}
    lens, page, heads = _lens(case), case["page"], h * case["group"]
    if case["op"] == "attend":
        b = sum(lens) * h * row * pools + sum(_ceil(x, page) for x in lens) * 4 + case["n_req"] * (heads * (4 * d + 4) + 4)
        return {"bytes": float(b), "flops": 4.0 * sum(lens) * heads * d}
    if case["op"] == "weigh":
        # keys in, weights in (unless they start anew) and out, queries and the softmax's denominators in
        b = sum(lens) * h * (row + (8 if case["decay"] else 4)) + sum(_ceil(x, page) for x in lens) * 4 + case["n_req"] * (heads * (2 * d + 4) + 4)
        return {"bytes": float(b), "flops": 2.0 * sum(lens) * heads * d}
    cut = [x for x in lens if x > case["limit"]]
    kept = len(cut) * case["keep"] * h
    # all weights in; kept rows, scales and weights in and out; which ones; pages back to the list
    b = sum(cut) * h * 4 + kept * (2 * row * pools + 4 + 4) + sum(_ceil(x, page) for x in cut) * 8 + case["n_req"] * 16
    if case["cache"] != "same":  # read back as values
        b += kept * pools * (row + 2 * d) + kept // h * 8
    return {"bytes": float(b), "flops": 0.0}


# ---- rows of 4 bits: 2688 = 6 x 448, the largest code times the largest block scale ----
def _quantise(x):
    """Codes [.., dim] (0 .. 15, the sign in bit 3), block scales [.., dim / 16] as e4m3 and row scales [..] of rows x in 32 bits.
    With rows of 16-bit types every quotient below is rounded once and keeps its side of a tie."""
    big = x.abs().amax(-1)
    blocks = x.unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    safe = torch.where(big == 0, 1.0, big)[..., None]
    scale = (top * 448.0 / safe).to(torch.float8_e4m3fn)
    s = scale.to(torch.float32)
    den = (safe * torch.where(s == 0, 1.0, s))[..., None]
    y = torch.where((s == 0)[..., None], 0.0, blocks.abs() * 2688.0 / den)
    code = (y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    code = code.to(torch.uint8) + (blocks < 0).to(torch.uint8) * 8
    return code.flatten(-2), scale, big / torch.full((), 2688.0, device=x.device)


def _levels(device):
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-v for v in half], device=device)


class _Pool:
    """A pool [page, head, token, ..] in the case's layout with its scales, and what a handle wants to know of it."""

    def __init__(self, case, n_pages, gen=None):
        self.kind, self.page, h, p, d = case["cache"], case["page"], case["kv_heads"], case["page"], case["dim"]
        self.dtype = _TYPES[case["dtype"]]
        shape = (n_pages, p, h) if case["layout"] == "token" else (n_pages, h, p)
        self.scale = self.block = self.record = None
        if self.kind == "fp4":
            x = torch.zeros(shape + (d // 2,), dtype=torch.uint8, device="cuda")
            self.record = torch.zeros((n_pages, h, p * (4 + d // 16)), dtype=torch.uint8, device="cuda")
            self.scale = self.record[:, :, :4 * p].view(torch.float32)
            self.block = self.record[:, :, 4 * p:].unflatten(-1, (p, d // 16))
        elif self.kind == "int8":
            x = torch.zeros(shape + (d,), dtype=torch.int8, device="cuda")
            self.record = self.scale = torch.rand((n_pages, h, p), generator=gen, device="cuda") * 0.03 + 0.01
        else:
            x = torch.zeros(shape + (d,), dtype=self.dtype, device="cuda")
        self.data = x.permute(0, 2, 1, 3) if case["layout"] == "token" else x
        if gen is None:
            return
        step = max(1, 30_000_000 // (h * p * d))  # normal rows, some pages at a time
        for i in range(0, n_pages, step):
            n = min(step, n_pages - i)
            rows = torch.randn((n, h, p, d), generator=gen, device="cuda")
            if self.kind == "fp4":
                code, block, scale = _quantise(rows.to(self.dtype).to(torch.float32))
                self.data[i:i + n] = code[..., ::2] + code[..., 1::2] * 16
                self.block[i:i + n] = block.view(torch.uint8)
                self.scale[i:i + n] = scale
            elif self.kind == "int8":
                self.data[i:i + n] = (rows * 40.0).round_().clamp_(-127, 127).to(torch.int8)
            else:
                self.data[i:i + n] = rows.to(self.dtype)

    def strides(self):
        return [x * (2 if self.kind == "fp4" else 1) for x in self.data.stride()[:3]]

    def values(self, page, head, at, to=torch.float32):
        """The values that rows (page, head, at) stand for."""
        x = self.data[page, head, at]
        if self.kind == "same":
            return x.to(to)
        scale = self.scale[page, head, at].to(to)[..., None]
        if self.kind == "int8":
            return x.to(to) * scale
        block = self.block[page, head, at].view(torch.float8_e4m3fn).to(to)
        code = torch.stack((x & 15, x >> 4), -1).flatten(-2).long()
        return (_levels(x.device).to(to)[code].unflatten(-1, (-1, 16)) * block[..., None]).flatten(-2) * scale

    def tensors(self):
        """What moves with a row: data, and scales."""
        return [t for t in (self.data, self.scale, self.block) if t is not None]


def _handle(case, n_pages, max_req, max_pages, k, v):
    import cvr_ranking_model_gb300 as cvr
    dt = {"bf16": cvr.DTYPE_BF16, "f16": cvr.DTYPE_F16}[case["dtype"]]

    def ptr(t):
        return 0 if t is None else t.data_ptr()

    cfg = cvr.make_kv_config(q_heads=case["kv_heads"] * case["group"], kv_heads=case["kv_heads"], head_dim=case["dim"], page_size=case["page"],
                             n_pages=n_pages, max_req=max_req, max_pages=max_pages, dtype=dt,
                             cache_dtype={"same": dt, "int8": cvr.DTYPE_I8, "fp4": cvr.DTYPE_FP4}[case["cache"]],
                             k=ptr(k.data), k_strides=k.strides(), k_scale=ptr(k.record),
                             v=0 if v is None else ptr(v.data), v_strides=() if v is None else v.strides(), v_scale=0 if v is None else ptr(v.record))
    return cvr.KvCache(cfg, torch.cuda.current_stream().cuda_stream)


# ---- inputs ----
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    (_prepare_rows if case["op"] in ("append", "read") else _prepare_requests)(case, s, gen)
    return s


def _prepare_rows(case, s, gen):
    n, h, d, page, dt = case["n_tok"], case["kv_heads"], case["dim"], case["page"], _TYPES[case["dtype"]]
    runs = _ceil(n, case["run"])  # runs of consecutive tokens, each in pages of its own from an offset of its own
    per = _ceil(case["run"] + page - 1, page)
    n_pages = runs * per + 3
    pages = torch.randperm(n_pages, generator=gen, device="cuda")[:runs * per].view(runs, per)
    i = torch.arange(n, device="cuda")
    r = i // case["run"]
    at = i % case["run"] + torch.randint(0, page, (runs,), generator=gen, device="cuda")[r]
    s["slots"] = pages[r, at // page] * page + at % page
    fill = gen if case["op"] == "read" else None
    s["k"] = _Pool(case, n_pages, fill)
    s["v"] = None if case["shared"] else _Pool(case, n_pages, fill)
    if case["op"] == "append":
        # the new rows are columns of a fused projection: query heads, then key heads, then value heads
        qkv = torch.randn((n, (case["group"] + 2) * h * d), generator=gen, device="cuda").to(dt)
        s["k_new"], s["v_new"] = qkv[:, case["group"] * h * d:(case["group"] + 1) * h * d], qkv[:, (case["group"] + 1) * h * d:]
    s["k_out"] = torch.empty((n, h, d), dtype=dt, device="cuda")
    s["v_out"] = None if case["shared"] else torch.empty_like(s["k_out"])
    if own:
        s["kv"] = _handle(case, n_pages, 1, 1, s["k"], s["v"])


def _prepare_requests(case, s, gen):
    n, lens, h, page = case["n_req"], _lens(case), case["kv_heads"], case["page"]
    max_pages = max(1, _ceil(case["max_len"], page))
    need = sum(_ceil(x, page) for x in lens)
    n_pages = need + need // 16 + 61
    perm = torch.randperm(n, generator=gen, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")[perm].contiguous()
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    count = (s["lens"].long() + page - 1) // page
    first, j = count.cumsum(0) - count, torch.arange(max_pages, device="cuda")
    at = (first[:, None] + j).clamp_(max=n_pages - 1)
    s["table"] = torch.where(j < count[:, None], order[at], -1).to(torch.int32)
    s["k"] = _Pool(case, n_pages, gen)
    s["v"] = None if case["shared"] else _Pool(case, n_pages, gen)
    heads = h * case["group"]
    s["scale"] = case["dim"] ** -0.5
    if case["op"] == "evict":
        # sums of attention weights: few heavy tokens, many light ones, some that no query ever saw
        w = torch.exp(torch.randn((n_pages, h, page), generator=gen, device="cuda") * 2.0)
        s["weight"] = torch.where(torch.rand((n_pages, h, page), generator=gen, device="cuda") < 0.1, 0.0, w)
        s["kept"] = torch.zeros((n, h, case["keep"]), dtype=torch.int32, device="cuda")
        s["lens_out"], s["pages"] = torch.empty_like(s["lens"]), torch.empty_like(s["lens"])
        # the list's first entries are in use: what is released takes their place
        s["free"], s["head"] = order.clone(), count.sum().to(torch.int32).reshape(1)
        s["head_out"] = torch.empty_like(s["head"])
        if case["cache"] != "same":  # 8 and 4 bits are compared as values: the slots of the kept rows, in order
            i = torch.arange(case["keep"], device="cuda")
            cut = s["table"][s["lens"] > case["limit"]].long()
            s["slots"] = (cut[:, i // page] * page + i % page).flatten().contiguous()
            s["k_out"] = torch.empty((s["slots"].numel(), h, case["dim"]), dtype=_TYPES[case["dtype"]], device="cuda")
            s["v_out"] = None if case["shared"] else torch.empty_like(s["k_out"])
    else:
        s["q"] = (torch.randn((n, heads, case["dim"]), generator=gen, device="cuda") * 2.0).to(_TYPES[case["dtype"]])
        if case["op"] == "weigh":
            s["lse"] = _softmax(case, s, torch.float32)[1].contiguous()  # as the attention of the same queries left it
            s["weight"] = torch.rand((n_pages, h, page), generator=gen, device="cuda")
        else:
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((n, heads), dtype=torch.float32, device="cuda")
    if own:
        s["kv"] = _handle(case, n_pages, n, max_pages, s["k"], s["v"])


# ---- one pass ----
def run(s):
    return {"append": _run_append, "read": _run_read, "attend": _run_attend, "weigh": _run_weigh, "evict": _run_evict}[s["case"]["op"]](s)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _read(s):
    """The rows of s["slots"] as values."""
    if own:
        s["kv"].read(s["slots"].numel(), s["slots"].data_ptr(), s["k_out"].data_ptr(), _ptr(s["v_out"]))
    else:
        page, at = s["slots"] // s["case"]["page"], s["slots"] % s["case"]["page"]
        for x in ("k", "v"):
            if s[x] is not None:
                s[x + "_out"] = s[x].values(page, slice(None), at).to(s["k_out"].dtype)
    return {x: s[x + "_out"] for x in ("k", "v") if s[x] is not None}


def _run_append(s):
    c = s["case"]
    if own:
        k, v = s["k_new"], s["v_new"]
        s["kv"].append(c["n_tok"], s["slots"].data_ptr(), k.data_ptr(), 0 if c["shared"] else v.data_ptr(), k_stride=k.stride(0), v_stride=v.stride(0))
    else:
        page, at = s["slots"] // c["page"], s["slots"] % c["page"]
        for x in ("k", "v"):
            if s[x] is not None:
                code, block, scale = _quantise(s[x + "_new"].to(torch.float32).unflatten(1, (c["kv_heads"], c["dim"])))
                s[x].data[page, :, at] = code[..., ::2] + code[..., 1::2] * 16
                s[x].block[page, :, at] = block.view(torch.uint8)
                s[x].scale[page, :, at] = scale
    return _read(s)


def _run_read(s):
    return _read(s)


def _softmax(case, s, to):
    """Of every request and query head the logits of its tokens and their log sum, in type `to`."""
    n, h = case["n_req"], case["kv_heads"]
    logits, lse = [], torch.full((n, h * case["group"]), float("-inf"), dtype=to, device="cuda")
    for r, length in enumerate(s["lens"].tolist()):
        j = torch.arange(length, device="cuda")
        k = s["k"].values(s["table"][r, j // case["page"]].long(), slice(None), j % case["page"], to)  # [token, head, dim]
        x = torch.matmul(s["q"][r].to(to).view(h, case["group"], -1), k.permute(1, 2, 0)) * s["scale"]
        logits.append(x)
        if length:
            top = x.amax(-1, keepdim=True)
            lse[r] = (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))).flatten()
    return logits, lse


def _gather(s, name):
    """All rows [request, head, token, dim] in 32 bits, those behind a history's end included."""
    at = s["table"].clamp(min=0).long()
    return s[name].values(at, slice(None), slice(None)).transpose(1, 2).flatten(2, 3)


def _logits(s):
    c = s["case"]
    k = _gather(s, "k")
    seen = (torch.arange(k.shape[2], device="cuda") < s["lens"].long()[:, None])[:, None, None, :]
    x = torch.matmul(s["q"].to(torch.float32).view(c["n_req"], c["kv_heads"], c["group"], -1), k.transpose(2, 3)) * s["scale"]
    return x, seen, k


def _run_attend(s):
    c = s["case"]
    if own:
        s["kv"].attend(c["n_req"], s["q"].data_ptr(), s["lens"].data_ptr(), s["table"].data_ptr(), s["scale"], s["out"].data_ptr(), lse=s["lse"].data_ptr())
        return {"out": s["out"], "lse": s["lse"]}
    x, seen, k = _logits(s)
    v = k if c["shared"] else _gather(s, "v")
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(x - safe)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v * seen.transpose(2, 3)) / torch.where(total == 0, 1.0, total)
    lse = safe + torch.log(total)
    return {"out": o.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(c["n_req"], -1)}


def _places(s):
    """Page and position of every place of every request's table, and which of them hold a token."""
    page = s["case"]["page"]
    j = torch.arange(s["table"].shape[1] * page, device="cuda")
    return s["table"][:, j // page].long(), j % page, j < s["lens"].long()[:, None]


def _run_weigh(s):
    c = s["case"]
    if own:
        s["kv"].weigh(c["n_req"], s["q"].data_ptr(), s["lens"].data_ptr(), s["table"].data_ptr(), s["scale"], s["lse"].data_ptr(), s["weight"].data_ptr(),
                      decay=c["decay"])
        return s["weight"]
    x, seen, _ = _logits(s)
    lse = s["lse"].view(c["n_req"], c["kv_heads"], c["group"], 1)
    p = torch.where(seen, torch.exp(x - lse), 0.0).sum(2).transpose(1, 2)  # [request, token, head]
    page, at, there = _places(s)
    at = at.expand_as(page)[there]
    page = page[there]
    newest = (torch.arange(there.shape[1], device="cuda") == s["lens"].long()[:, None] - 1)[there][:, None]
    before = torch.where(newest, 0.0, s["weight"][page, :, at] * c["decay"])
    s["weight"][page, :, at] = before + p[there]
    return s["weight"]


def _run_evict(s):
    c = s["case"]
    page, keep = c["page"], c["keep"]
    if own:
        s["kv"].evict(c["n_req"], s["lens"].data_ptr(), c["limit"], keep, s["table"].data_ptr(), s["weight"].data_ptr(), s["kept"].data_ptr(),
                      s["lens_out"].data_ptr(), first=c["first"], last=c["last"], pages=s["pages"].data_ptr(), free_pages=s["free"].data_ptr(),
                      n_free=s["free"].numel(), free_head=s["head"].data_ptr(), free_head_out=s["head_out"].data_ptr())
    else:
        lens = s["lens"].long()
        cut = lens > c["limit"]
        rows, n = s["table"][cut].long(), lens[cut][:, None]
        j = torch.arange(rows.shape[1] * page, device="cuda")
        w = s["weight"][rows[:, j // page], :, j % page]  # [request, token, head]
        must = (j < c["first"]) | (j >= n - c["last"])
        w = torch.where(must[..., None], float("inf"), w)
        w = torch.where((j < n)[..., None], w, float("-inf"))
        best = torch.sort(w.transpose(1, 2), dim=2, descending=True, stable=True).indices[:, :, :keep]
        kept = torch.sort(best, dim=2).values  # [request, head, place]
        i, h = torch.arange(keep, device="cuda"), torch.arange(c["kv_heads"], device="cuda")[:, None]
        r = torch.arange(rows.shape[0], device="cuda")[:, None, None]
        source, target = rows[r, kept // page], rows[r, i // page]
        moved = [s["weight"]] + s["k"].tensors() + (s["v"].tensors() if s["v"] is not None else [])
        for x in moved:
            x[target, h, i % page] = x[source, h, kept % page]
        s["kept"][cut] = kept.to(torch.int32)
        s["lens_out"] = torch.where(cut, keep, lens).to(torch.int32)
        held = (lens + page - 1) // page
        left = torch.where(cut, _ceil(keep, page), held)
        s["pages"] = left.to(torch.int32)
        e = torch.arange(s["table"].shape[1], device="cuda")
        back = s["table"][(e >= left[:, None]) & (e < held[:, None])]
        s["head_out"] = s["head"] - back.numel()
        s["free"][s["head_out"] + torch.arange(back.numel(), device="cuda")] = back
    res = {"kept": s["kept"], "lens": s["lens_out"], "pages": s["pages"], "free": s["free"], "head": s["head_out"], "weight": s["weight"]}
    if c["cache"] != "same":
        res.update(_read(s))
    else:
        res.update({x: s[x].data for x in ("k", "v") if s[x] is not None})
    return res


# ---- the definition in 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](case, s)


def _nearest(x, levels):
    """The nearest of rising levels, the one at an even place where two are as near."""
    i = torch.searchsorted(levels, x).clamp_(max=levels.numel() - 1)
    low = (i - 1).clamp_(min=0)
    a, b = x - levels[low], levels[i] - x
    return levels[torch.where((a < b) | ((a == b) & (low % 2 == 0)), low, i)]


def _exact_append(case, s):
    e2m1 = _levels("cuda")[:8].double()
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    res = {}
    for x in ("k", "v"):
        if s[x] is None:
            continue
        new = s[x + "_new"].double().unflatten(1, (case["kv_heads"], -1, 16))  # [token, head, block, 16]
        big = new.abs().flatten(2).max(dim=2).values[:, :, None, None].clamp(min=1e-300)
        block = _nearest(new.abs().max(dim=3, keepdim=True).values * 448.0 / big, e4m3)
        code = _nearest((new.abs() * 2688.0 / (big * block.clamp(min=1e-300))).clamp(max=6.0), e2m1)
        res[x] = (torch.sign(new) * code * block * big / 2688.0).flatten(2)
    return res


def _one_row(case, s, name, r, h, length):
    """A history's rows of one head in 64 bits, from the bits of their pages."""
    pool, ids, d = s[name], s["table"][r, :_ceil(length, case["page"])].long(), case["dim"]
    x = pool.data[ids, h].flatten(0, 1)[:length]
    if case["cache"] == "same":
        return x.double()
    scale = pool.scale[ids, h].flatten()[:length, None].double()
    if case["cache"] == "int8":
        return x.double() * scale
    value = torch.zeros((length, d), dtype=torch.float64, device="cuda")
    for odd in (0, 1):
        c = (x >> 4 if odd else x & 15).long()
        m, e = (c & 1).double(), c >> 1 & 3
        size = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * 2.0 ** (e - 1).double())
        value[:, odd::2] = torch.where(c > 7, -size, size)
    b = pool.block[ids, h].flatten(0, 1)[:length].long()
    m, e = (b & 7).double(), b >> 3 & 15
    block = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7).double())
    return value * block.repeat_interleave(16, dim=1) * scale


def _exact_read(case, s):
    res = {}
    pages = torch.arange(s["k"].data.shape[0], device="cuda")
    whole = dict(s, table=pages[None])
    for x in ("k", "v"):
        if s[x] is not None:
            rows = [_one_row(case, whole, x, 0, h, pages.numel() * case["page"])[s["slots"]] for h in range(case["kv_heads"])]
            res[x] = torch.stack(rows, 1)
    return res


def _exact_attend(case, s):
    g = case["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lens"].tolist()):
        for h in range(case["kv_heads"] if n else 0):
            k = _one_row(case, s, "k", r, h, n)
            v = k if case["shared"] else _one_row(case, s, "v", r, h, n)
            x = s["q"][r, h * g:(h + 1) * g].double() @ k.T * s["scale"]
            out[r, h * g:(h + 1) * g] = torch.softmax(x, dim=1) @ v
            lse[r, h * g:(h + 1) * g] = torch.logsumexp(x, dim=1)
    return {"out": out, "lse": lse}


def _exact_weigh(case, s):
    g, page, weight = case["group"], case["page"], s["weight"].double()
    for r, n in enumerate(s["lens"].tolist()):
        for h in range(case["kv_heads"] if n else 0):
            x = s["q"][r, h * g:(h + 1) * g].double() @ _one_row(case, s, "k", r, h, n).T * s["scale"]
            p = torch.exp(x - s["lse"][r, h * g:(h + 1) * g, None].double()).sum(0)
            j = torch.arange(n, device="cuda")
            at = (s["table"][r].long()[j // page], h, j % page)
            old = weight[at] * case["decay"]
            old[-1] = 0.0
            weight[at] = old + p
    return weight


def _exact_evict(case, s):
    page, keep, table, head = case["page"], case["keep"], s["table"].tolist(), int(s["head"])
    lens = s["lens"].tolist()
    cut = [n > case["limit"] for n in lens]
    i, back = torch.arange(keep, device="cuda"), []
    for r, n in enumerate(lens):
        if not cut[r]:
            continue
        t, j = s["table"][r].long(), torch.arange(n, device="cuda")
        for h in range(case["kv_heads"]):
            w = s["weight"][t[j // page], h, j % page]
            w[:case["first"]] = float("inf")
            w[n - case["last"]:] = float("inf")
            least = torch.kthvalue(w, n - keep + 1).values
            stay = w > least
            ties = (w == least).nonzero().flatten()[:keep - int(stay.sum())]
            stay[ties] = True
            kept = stay.nonzero().flatten()
            s["kept"][r, h] = kept.to(torch.int32)
            for x in [s["weight"]] + s["k"].tensors() + (s["v"].tensors() if s["v"] is not None else []):
                x[t[i // page], h, i % page] = x[t[kept // page], h, kept % page].clone()
        back += table[r][_ceil(keep, page):_ceil(n, page)]
    s["free"][head - len(back):head] = torch.tensor(back, dtype=torch.int32, device="cuda")
    res = {"kept": s["kept"], "lens": [keep if x else n for x, n in zip(cut, lens)], "pages": [_ceil(keep if x else n, page) for x, n in zip(cut, lens)],
           "free": s["free"], "head": [head - len(back)], "weight": s["weight"].double()}
    res = {k: torch.tensor(v, dtype=torch.int32, device="cuda") if isinstance(v, list) else v for k, v in res.items()}
    if case["cache"] != "same":
        return {**res, **_exact_read(case, s)}
    return {**res, **{x: s[x].data.double() for x in ("k", "v") if s[x] is not None}}
