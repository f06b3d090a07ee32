"""Paged caches and 64-bit references shared by the tests of the target's cache and attention."""
import math

import torch

import speculative_decoding_verification_21_gb300 as sv

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest step
E4M3 = torch.float8_e4m3fn


def pow2(e):
    """2^e in float64, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def quantise64(x):
    """(code values in float64, scale bytes) of rows [..., D]: the definition, in 64 bits."""
    x = x.double()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    m, e = torch.frexp(fin.amax(-1) / 448.0)
    k = torch.where(m == 0.5, e - 1, e).clamp_min(-120)
    k = torch.where(fin.amax(-1) == 0, torch.full_like(k, -120), k)
    y = x / pow2(k)[..., None]
    step = pow2(torch.frexp(torch.where(torch.isfinite(y), y, 1.0).abs().clamp_min(2.0 ** -6))[1] - 4)
    code = torch.round(y / step) * step
    code = torch.where(torch.isfinite(x), code, math.nan)
    return code, (k + 127).to(torch.uint8)


class Case:
    """A pool, B sequences over shuffled pages of it, and packed rows for their chunks.

    lens: (new tokens, cached length with them) per sequence.  Everything a call must not read
    (slots behind a sequence's end, pages of nobody) holds NaN; table entries behind the last
    page are far out of range."""

    def __init__(self, lens, *, kv_heads=2, group=4, dim=64, page=16, dtype=torch.bfloat16,
                 cache=None, layout="hnd", seed=0, spare=3, device="cuda", scale_spread=0,
                 first_page=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.lens, self.H, self.G, self.D, self.ps = lens, kv_heads, group, dim, page
        self.dtype, self.cache_dtype = dtype, cache or dtype
        B = len(lens)
        need = [-(-max(L, 0) // page) for _, L in lens]
        self.pages = sum(need) + spare + first_page
        width = max(need + [1]) + 1
        order = (torch.randperm(sum(need) + spare, generator=g, device=device) + first_page).tolist()
        self.owned = []
        table = torch.full((B, width), 2 ** 30, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.owned.append(order[at:at + need[b]])
            table[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
            at += need[b]
        self.table = table.to(device)
        start = [0]
        for n, _ in lens:
            start.append(start[-1] + n)
        self.start_list, self.total = start, start[-1]
        self.start = torch.tensor(start, dtype=torch.int32, device=device)
        self.len = torch.tensor([L for _, L in lens], dtype=torch.int32, device=device)
        # keys and values of every position, then scattered into the pages
        shape = (self.pages, kv_heads, page, dim) if layout == "hnd" else (self.pages, page, kv_heads, dim)
        e4m3 = self.cache_dtype == E4M3
        self.k64, self.v64, pools, scales = [], [], [], []
        for store in (self.k64, self.v64):
            if first_page:  # most of the pool is never touched: leave it as it comes
                pool = torch.empty(shape, dtype=self.cache_dtype, device=device)
            else:
                pool = torch.full(shape, 255 if e4m3 else math.nan, device=device,
                                  dtype=torch.uint8 if e4m3 else self.cache_dtype)
                pool = pool.view(self.cache_dtype)
            pool = pool if layout == "hnd" else pool.transpose(1, 2)
            scale = torch.full((self.pages, kv_heads, page), 255, dtype=torch.uint8, device=device)
            for b, (n, L) in enumerate(lens):
                L = max(L, 0)
                x = torch.randn((L, kv_heads, dim), generator=g, device=device)
                if scale_spread:
                    x = x * 2.0 ** torch.randint(-scale_spread, scale_spread + 1, (L, kv_heads, 1),
                                                 generator=g, device=device)
                j = torch.arange(L, device=device)
                p = torch.tensor(self.owned[b] + [0], device=device)[j // page]
                if e4m3:
                    code, s = quantise64(x)
                    held = (code * pow2(s.int() - 127)[..., None])
                    pool.view(torch.uint8)[p, :, j % page] = code.float().to(E4M3).view(torch.uint8)
                    scale[p, :, j % page] = s
                    store.append(held.to(dtype).double())  # dequantised to the queries' type
                else:
                    x = x.to(self.cache_dtype)
                    pool[p, :, j % page] = x
                    store.append(x.double())
            pools.append(pool)
            scales.append(scale if e4m3 else None)
        self.cache = sv.KVCache(pools[0], pools[1], scales[0], scales[1])
        # queries as a slice of a wider projection: neither stride is the packed one
        wide = torch.randn((self.total, kv_heads * group + 3, dim + 16), generator=g, device=device)
        self.q = (wide * 1.5).to(dtype)[:, 1:1 + kv_heads * group, :dim]

    def reference(self, window=0, scale=None):
        """(out, lse, bound on |error| of out, of lse) in float64."""
        scale = self.D ** -0.5 if scale is None else scale
        outs, lses, tols, ltols = [], [], [], []
        half, tiny = HALF[self.dtype], TINY[self.dtype]
        for b, (n, L) in enumerate(self.lens):
            if n == 0:
                continue
            q = self.q[self.start_list[b]:self.start_list[b + 1]].double()
            q = q.reshape(n, self.H, self.G, self.D)
            k, v = self.k64[b], self.v64[b]
            s = torch.einsum("nhgd,lhd->nhgl", q, k) * scale
            at = L - n + torch.arange(n, device=q.device)
            j = torch.arange(k.shape[0], device=q.device)
            seen = j <= at[:, None]
            if window:
                seen = seen & (j > at[:, None] - window)
            s = s.masked_fill(~seen[:, None, None], -math.inf)
            lse = torch.logsumexp(s, -1) if k.shape[0] else s.new_full(s.shape[:-1], -math.inf)
            p = torch.exp(s - lse[..., None]).nan_to_num(0.0) if k.shape[0] else s
            o = torch.einsum("nhgl,lhd->nhgd", p, v)
            mass = torch.einsum("nhgl,lhd->nhgd", p, v.abs())
            # a score: head_dim products summed in fp32, times the scale, minus the maximum
            # (log2 units), and an exponential good to 2 ulp
            big = (torch.einsum("nhgd,lhd->nhgl", q.abs(), k.abs()) * abs(scale)).amax(-1) \
                if k.shape[0] else torch.zeros_like(lse)
            delta = ((self.D + 8) * big + 8) * 2.0 ** -24
            # sums of L terms in fp32, in any order: L 2^-24 at worst
            delta = delta + L * 2.0 ** -24
            # p rounded to the type once, the output once
            tol = half * o.abs() + (half + 2 * delta[..., None]) * mass * (1 + half) + tiny
            outs.append(o.reshape(n, -1, self.D))
            lses.append(lse.reshape(n, -1))
            tols.append(tol.reshape(n, -1, self.D))
            ltols.append((2 * delta + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22).reshape(n, -1))
        return torch.cat(outs), torch.cat(lses), torch.cat(tols), torch.cat(ltols)

    def attend(self, **kw):
        return sv.spec_chunk_attention(self.q, self.cache, self.table, self.start, self.len, **kw)

    def check(self, window=0, scale=None, **kw):
        o = self.attend(window=window, scale=scale, want_flags=True, **kw)
        out, lse, tol, ltol = self.reference(window, scale)
        torch.cuda.synchronize()
        err = (o["out"].double() - out).abs()
        assert bool((err <= tol).all()), \
            f"out off by {float((err / tol).nan_to_num(math.inf).max()):.2f} of its bound"
        empty = torch.isinf(lse)
        assert torch.equal(torch.isneginf(o["lse"]), empty), "empty rows"
        lerr = (o["lse"].double() - lse).abs().masked_fill(empty, 0.0)
        assert bool((lerr <= ltol).all()), f"lse off by {float((lerr / ltol).max()):.2f} of its bound"
        assert not bool(o["flags"].any())
        return o
