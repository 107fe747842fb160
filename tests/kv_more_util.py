"""Helpers of the tests of 4-bit pools, of rows read back, attention weights and eviction: caches with 4-bit pools and the
operators' definitions in 64 bits."""
from __future__ import annotations

import math

from kv_util import EPS, Cache, cvr_type, fill_rubbish, pool

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # e2m1


def e4m3_values():
    """The finite e4m3 numbers >= 0 in 64 bits, by their code 0 .. 126."""
    return [(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def nearest(x, levels):
    """Places of the nearest of rising levels (even places where two are as near) for x >= 0 in 64 bits, beyond the last: the last."""
    import torch
    lv = torch.tensor(levels, dtype=torch.float64, device=x.device)
    i = torch.searchsorted(lv, x).clamp_(max=len(levels) - 1)
    low = (i - 1).clamp_(min=0)
    a, b = x - lv[low], lv[i] - x
    return torch.where((a < b) | ((a == b) & (low % 2 == 0)), low, i)


def quantised(x):
    """Codes [.., dim] (0 .. 15), block scale codes [.., dim / 16] and row scales [..] (fp32) that cvr_kv_append makes of finite rows x.
    No quotient is closer than 2^-18 of it to a tie without being it, and ties are numbers of 64 bits: the roundings are the exact
    quotients'."""
    import torch
    x = x.double()
    big = x.abs().amax(-1)
    safe = torch.where(big == 0, 1.0, big)
    blocks = x.unflatten(-1, (-1, 16))
    scale = nearest(448.0 * blocks.abs().amax(-1) / safe[..., None], e4m3_values())
    s = torch.tensor(e4m3_values(), dtype=torch.float64, device=x.device)[scale]
    y = torch.where((s == 0)[..., None], 0.0, 2688.0 * blocks.abs() / (safe[..., None] * torch.where(s == 0, 1.0, s))[..., None])
    code = nearest(y, LEVELS) + 8 * (torch.signbit(blocks)).long()
    return code.flatten(-2).to(torch.uint8), scale.to(torch.uint8), (big.float() / torch.full((), 2688.0, device=x.device))


def value_of(code, scale, row_scale):
    """What codes (uint8 [.., dim]), block scale codes and row scales stand for, in 64 bits."""
    import torch
    lv = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=code.device)[code.long()]
    e = torch.tensor(e4m3_values() + [math.nan], dtype=torch.float64, device=code.device)[(scale & 127).long()]
    e = torch.where(scale > 127, -e, e)
    return (lv.unflatten(-1, (-1, 16)) * e[..., None]).flatten(-2) * row_scale.double()[..., None]


class Pool4:
    """A pool of 4 bits: codes [page, head, token, dim / 2] in a layout, and records with views of their two parts."""

    def __init__(self, n_pages, heads, page, dim, layout):
        import torch
        self.codes = pool(n_pages, heads, page, dim // 2, "i8", layout).view(torch.uint8)
        self.record = torch.empty((n_pages, heads, page * (4 + dim // 16)), dtype=torch.uint8, device="cuda")
        self.scale = self.record[:, :, :4 * page].view(torch.float32)
        self.block = self.record[:, :, 4 * page:].unflatten(-1, (page, dim // 16))

    def strides(self):
        return [2 * x for x in self.codes.stride()[:3]]

    def unpacked(self, *at):
        import torch
        x = self.codes[at]
        return torch.stack((x & 15, x >> 4), -1).flatten(-2)

    def values(self, *at):
        return value_of(self.unpacked(*at), self.block[at], self.scale[at])

    def put(self, at, code, block, scale):
        self.codes[at] = code[..., ::2] + code[..., 1::2] * 16
        self.block[at] = block
        self.scale[at] = scale


class Cache4(Cache):
    """A cache whose pools are 4 bits (k and v are Pool4), 8 bits or 16: rubbish behind the histories, NaN scales among it."""

    def __init__(self, *args, cache="fp4", **kw):
        self.form = cache
        super().__init__(*args, cache="same" if cache == "fp4" else cache, **kw)

    def _pool(self, layout, spread):
        import torch
        if self.form != "fp4":
            return super()._pool(layout, spread)
        p = Pool4(self.n_pages, self.heads, self.page, self.dim, layout)
        p.codes.copy_(torch.randint(0, 256, p.codes.shape, generator=self.gen, device="cuda"))
        p.block.copy_(torch.randint(0, 256, p.block.shape, generator=self.gen, device="cuda"))
        p.block[..., 0] = 127  # NaN
        p.scale.fill_(math.nan)
        for r, n in enumerate(self.lens_list):
            for j in range(0, n, self.page):
                m, at = min(self.page, n - j), int(self.table[r, j // self.page])
                p.codes[at, :, :m] = torch.randint(0, 256, p.codes[at, :, :m].shape, generator=self.gen, device="cuda").to(torch.uint8)
                p.block[at, :, :m] = torch.randint(0, 127, p.block[at, :, :m].shape, generator=self.gen, device="cuda").to(torch.uint8)
                p.scale[at, :, :m] = torch.rand((self.heads, m), generator=self.gen, device="cuda") * (spread * 4 / 2688)
        return p, None

    def handle(self, q_heads, window=0, stream=0, max_req=None):
        import cvr_ranking_model_gb300 as cvr
        if self.form != "fp4":
            return super().handle(q_heads, window, stream, max_req)
        v = self.v
        cfg = cvr.make_kv_config(q_heads, self.heads, self.dim, self.page, self.n_pages, max_req or max(1, len(self.lens_list)), self.max_pages,
                                 cvr_type(self.dtype), cvr.DTYPE_FP4, window, self.k.codes.data_ptr(), self.k.strides(), self.k.record.data_ptr(),
                                 0 if v is None else v.codes.data_ptr(), () if v is None else v.strides(), 0 if v is None else v.record.data_ptr())
        return cvr.KvCache(cfg, stream)

    def rows(self, r, head, lo, hi):
        import torch
        if self.form != "fp4":
            return super().rows(r, head, lo, hi)
        j = torch.arange(lo, hi, device="cuda")
        p = self.table[r].long()[j // self.page]
        k = self.k.values(p, head, j % self.page)
        return [k, k if self.v is None else self.v.values(p, head, j % self.page)]

    def stored(self):
        """Every tensor that holds rows or scales, as [page, head, token, ..]."""
        if self.form == "fp4":
            return [t for p in (self.k, self.v) if p is not None for t in (p.codes, p.block, p.scale)]
        return [t for t in (self.k, self.k_scale, self.v, self.v_scale) if t is not None]

    def slots(self, r, tokens):
        """Slots of a request's tokens."""
        return self.table[r].long()[tokens // self.page] * self.page + tokens % self.page

    def weigh_reference(self, q, scale, lse, weight, decay, new):
        """(weight, bound) in 64 bits after cvr_kv_weigh. To first order a weight p = exp(x - lse) is off by
          - the logit x: its D exact products' sum at most D 2^-23 of sum |q k| scale, the products with the row's scale and the
            factor a rounding each; queries held in fp16 (bf16 ones on 8 and 4 bits) 2^-25 of their largest value per value;
          - the difference's rounding, the product with log2 e and its constant, 2^-24 of |x - lse| each; exp2 2^-21;
        the sum over the heads loses 2^-24 per addend, and the old weight's part and the sum of both 2^-24 each."""
        import torch
        ref, bound = weight.double().clone(), torch.zeros(weight.shape, dtype=torch.float64, device="cuda")
        g = q.shape[1] // self.heads
        for r in range(q.shape[0]):
            n = min(max(self.lens_list[r], 0), self.max_pages * self.page)
            if n == 0:
                continue
            j = torch.arange(n, device="cuda")
            page, at = self.table[r].long()[j // self.page], j % self.page
            for h in range(self.heads):
                k, _ = self.rows(r, h, 0, n)
                x = q[r, h * g:(h + 1) * g].double()
                s, size = x @ k.T * scale, x.abs() @ k.abs().T * abs(scale)
                d = s - lse[r, h * g:(h + 1) * g, None].double()
                p = torch.exp(d)
                held = 0.0
                if self.dtype == "bf16" and self.form != "same":
                    held = x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] * abs(scale) * 2.0 ** -25
                off = size * self.dim * 2.0 ** -23 + s.abs() * 3 * 2.0 ** -24 + d.abs() * 3 * 2.0 ** -24 + held + 2.0 ** -21
                old = torch.where(j < n - new[r], weight[page, h, at].double() * decay, 0.0) if decay else torch.zeros_like(p[0])
                total = old + p.sum(0)
                ref[page, h, at] = total
                bound[page, h, at] = (p * (off + g * 2.0 ** -24)).sum(0) + total.abs() * 2 * 2.0 ** -24 + 2.0 ** -140
        return ref, bound


def evict_reference(c, lens, limit, keep, first, last, weight, table, page):
    """kept {(r, h): tensor}, lens after; ties and NaN by the definition."""
    import torch
    kept = {}
    for r, n in enumerate(lens):
        if n <= limit:
            continue
        j = torch.arange(n, device="cuda")
        for h in range(c.heads):
            w = weight[table[r].long()[j // page], h, j % page].double()
            w = torch.where(torch.isnan(w), -math.inf, w) + 0.0
            nan = torch.isnan(weight[table[r].long()[j // page], h, j % page])
            mid = list(range(first, n - last))
            wl, nl = w.tolist(), nan.tolist()
            mid.sort(key=lambda i: (nl[i], -wl[i], i))
            chosen = sorted(mid[:keep - first - last])
            kept[r, h] = torch.tensor(list(range(first)) + chosen + list(range(n - last, n)), dtype=torch.int32, device="cuda")
    return kept, [keep if n > limit else n for n in lens]


__all__ = ["EPS", "Cache4", "Pool4", "quantised", "value_of", "evict_reference", "fill_rubbish", "e4m3_values"]
