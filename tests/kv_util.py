"""Helpers of the paged history cache's tests: pools of any layout with rubbish in every place that must not be read,
and the operators' definitions in 64 bits and in plain integers."""
from __future__ import annotations

import math

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step of a rounding, relative to the value


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}[name]


def cvr_type(name):
    import cvr_ranking_model_gb300 as cvr
    return {"bf16": cvr.DTYPE_BF16, "f16": cvr.DTYPE_F16, "i8": cvr.DTYPE_I8}[name]


def pool(n_pages, heads, page, dim, kind, layout):
    """An uninitialised pool seen as [page, head, token, dim]. Layouts: "page" [page][head][token], "token"
    [page][token][head], "gaps" [head][page][token] with unused values after every row and page."""
    import torch
    t = torch_type(kind)
    if layout == "token":
        return torch.empty((n_pages, page, heads, dim), dtype=t, device="cuda").permute(0, 2, 1, 3)
    if layout == "gaps":
        return torch.empty((heads, n_pages, page + 1, dim + 32), dtype=t, device="cuda").permute(1, 0, 2, 3)[:, :, :page, :dim]
    return torch.empty((n_pages, heads, page, dim), dtype=t, device="cuda")


def fill_rubbish(x, gen):
    """Values that ruin any sum they enter."""
    import torch
    if x.dtype == torch.int8:
        x.copy_(torch.randint(-128, 128, x.shape, generator=gen, device="cuda"))
        return
    if x.numel() > 2 ** 30:
        x.fill_(math.nan)
        return
    bad = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(x.dtype).max, torch.finfo(x.dtype).min], device="cuda")
    x.copy_(bad[torch.randint(0, 5, x.shape, generator=gen, device="cuda")].to(x.dtype))


class Cache:
    """Pools that hold `lens` tokens per request (values of unit size times `spread`), the rest rubbish."""

    def __init__(self, lens, heads, dim, page, dtype="bf16", cache="same", layout="page", shared=False, seed=0, max_pages=None,
                 spread=1.0, spare=5):
        import torch
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gen, self.lens_list, self.heads, self.dim, self.page, self.dtype = gen, list(lens), heads, dim, page, dtype
        self.kind = "i8" if cache == "i8" else dtype
        self.shared = shared
        need = [-(-max(0, n) // page) for n in lens]
        self.max_pages = max_pages or max(1, max(need, default=1)) + 2
        self.n_pages = sum(need) + spare
        self.lens = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
        order = torch.randperm(self.n_pages, generator=gen, device="cuda").to(torch.int32)
        # entries behind a request's pages: ids that must not be followed
        self.table = torch.randint(-2 ** 31, 2 ** 31 - 1, (max(1, len(need)), self.max_pages), generator=gen, device="cuda").to(torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.k, self.k_scale = self._pool(layout, spread)
        self.v, self.v_scale = (None, None) if shared else self._pool(layout, spread)

    def _pool(self, layout, spread):
        import torch
        x = pool(self.n_pages, self.heads, self.page, self.dim, self.kind, layout)
        fill_rubbish(x, self.gen)
        scale = None
        if self.kind == "i8":
            scale = torch.full((self.n_pages, self.heads, self.page), math.nan, device="cuda")
        for r, n in enumerate(self.lens_list):
            for j in range(0, n, self.page):
                m, p = min(self.page, n - j), int(self.table[r, j // self.page])
                val = torch.randn((self.heads, m, self.dim), generator=self.gen, device="cuda") * spread
                if scale is None:
                    x[p, :, :m] = val.to(x.dtype)
                else:
                    x[p, :, :m] = (val * 40).round().clamp(-127, 127).to(torch.int8)
                    scale[p, :, :m] = torch.rand((self.heads, m), generator=self.gen, device="cuda") * 0.05
        return x, scale

    def handle(self, q_heads, window=0, stream=0, max_req=None):
        import cvr_ranking_model_gb300 as cvr

        def ptr(t):
            return 0 if t is None else t.data_ptr()

        cfg = cvr.make_kv_config(q_heads, self.heads, self.dim, self.page, self.n_pages, max_req or max(1, len(self.lens_list)),
                                 self.max_pages, cvr_type(self.dtype), cvr_type(self.kind), window, ptr(self.k), self.k.stride()[:3],
                                 ptr(self.k_scale), ptr(self.v), () if self.v is None else self.v.stride()[:3], ptr(self.v_scale))
        return cvr.KvCache(cfg, stream)

    def rows(self, r, head, lo, hi):
        """Keys and values of tokens lo..hi - 1 in 64 bits."""
        import torch
        res = []
        for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            if x is None:
                res.append(res[0])
                continue
            j = torch.arange(lo, hi, device="cuda")
            p = self.table[r].long()[j // self.page]
            t = x[p, head, j % self.page].double()
            res.append(t if s is None else t * s[p, head, j % self.page].double()[:, None])
        return res

    def reference(self, q, scale, window=0):
        """(out, lse, bound of out, bound of lse) in 64 bits for q [n_req, q_heads, dim].

        The bounds count, to first order, what an fp32 evaluation on the tensor cores may lose:
          - a logit: its D products are exact, their sum loses at most D 2^-23 of sum |q k| scale (adds that cut off), and
            the scalings and the exponent's argument 4 roundings of |s|; a weight's relative error is that, plus 2^-21 for
            exp2 and 2^-15 for its split into two 16-bit halves;
          - weights enter the numerator and the denominator: twice that, relative to sum p |v|;
          - the sums over tokens: one add per 16 tokens and 64 for the joins, 2^-23 each;
          - the output's rounding to its type (half a step, and half of the smallest subnormal)."""
        import torch
        n, heads, dim = q.shape
        g = heads // self.heads
        out = torch.zeros((n, heads, dim), dtype=torch.float64, device="cuda")
        lse = torch.full((n, heads), -math.inf, dtype=torch.float64, device="cuda")
        b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
        for r in range(n):
            hi = min(max(self.lens_list[r], 0), self.max_pages * self.page)
            lo = max(0, hi - window) if window else 0
            if hi == 0:
                continue
            for h in range(self.heads):
                k, v = self.rows(r, h, lo, hi)
                x = q[r, h * g:(h + 1) * g].double()
                s = x @ k.T * scale
                p = torch.softmax(s, 1)
                o = p @ v
                out[r, h * g:(h + 1) * g] = o
                lse[r, h * g:(h + 1) * g] = torch.logsumexp(s, 1)
                logit = (x.abs() @ k.abs().T * abs(scale)).amax(1, keepdim=True) * dim * 2.0 ** -23 + s.abs().amax(1, keepdim=True) * 4 * 2.0 ** -24
                sums = ((hi - lo) / 16 + 64) * 2.0 ** -23
                b_out[r, h * g:(h + 1) * g] = EPS[self.dtype] * o.abs() + (2 * (logit + 2.0 ** -21 + 2.0 ** -15) + 2 * sums) * (p @ v.abs()) + 2.0 ** -25
                b_lse[r, h * g:(h + 1) * g] = (logit + 2.0 ** -21 + sums)[:, 0] + lse[r, h * g:(h + 1) * g].abs() * 2.0 ** -22
        return out, lse, b_out, b_lse


def assert_within(got, ref, bound, what):
    import torch
    same = (got.double() == ref) | (torch.isnan(got) & torch.isnan(ref))
    off = torch.where(same, 0.0, (got.double() - ref).abs())
    bad = ~(off <= bound)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, the first at {at}: "
                             f"{float(got[at])} for {float(ref[at])}, bound {float(bound[at]):.3e}")


def tables_reference(lens, new, held, free, head, table, page, n_slots):
    """cvr_kv_tables in plain integers, for valid inputs: (table, pages, head, slots)."""
    table = [list(row) for row in table]
    pages, slots, at = [], [], head
    for r, n in enumerate(lens):
        need, have = -(-n // page), held[r]
        for j in range(have, need):
            table[r][j] = free[at] if at < len(free) else -1
            have += at < len(free)
            at += 1
        pages.append(max(have, held[r]))
        for pos in range(n - new[r], n):
            p = table[r][pos // page]
            slots.append(p * page + pos % page if p >= 0 else -1)
    slots = (slots + [-1] * n_slots)[:n_slots]
    return table, pages, min(at, len(free)), slots
