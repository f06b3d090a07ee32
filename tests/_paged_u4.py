"""Paged caches of 4-bit codes and 64-bit references, shared by their tests."""
import math

import torch

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import Case, HALF, TINY

BF, FP, U4 = torch.bfloat16, torch.float16, torch.uint8
NAN_WORD = 0x7FFF


def codes_of(x):
    """(codes uint8 [..., D], step and zero bf16 [..., 2]) of rows [..., D] by the definition: fp32
    operations, each rounded."""
    x = x.float()
    lo, hi = x.amin(-1), x.amax(-1)  # (NaN if there is one)
    z = lo.to(BF)
    half = z.float() * 0.5
    s = ((hi * 0.5 - half) * torch.tensor(2.0 / 15.0, device=x.device)).to(BF)
    s = torch.maximum(s, torch.tensor(2.0 ** -120, dtype=BF, device=x.device))
    c = torch.round((x * 0.5 - half[..., None]) / (s.float() * 0.5)[..., None]).clamp(0, 15)
    bad = ~(torch.isfinite(lo) & torch.isfinite(hi) & torch.isfinite(z) & torch.isfinite(s))
    c = torch.where(bad[..., None], torch.zeros_like(c), c)
    sz = torch.stack([s, z], -1)
    return c.to(torch.uint8), torch.where(bad[..., None], torch.full_like(sz, math.nan), sz)


def packed(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpacked(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def values(c, sz):
    """What codes stand for, in float64 (exact)."""
    sz = sz.double()
    return c.double() * sz[..., :1] + sz[..., 1:]


def pool_u4(pages, kv_heads, page, dim, layout, device="cuda", fill=0xA5):
    """An uninitialised-looking pool: arbitrary codes, steps and zeros NaN."""
    shape = (pages, kv_heads, page, dim // 2) if layout == "hnd" else (pages, page, kv_heads, dim // 2)
    pool = torch.full(shape, fill, dtype=torch.uint8, device=device)
    sz = torch.full((pages, kv_heads, page, 2), math.nan, dtype=BF, device=device)
    return (pool if layout == "hnd" else pool.transpose(1, 2)), sz


class CaseU4(Case):
    """tests._paged.Case over a cache of 4-bit codes.  What a call must not read holds NaN steps and
    zeros (a code by itself is never NaN)."""

    weight = 2.0 ** -11  # what a weight may be off by, relative: an fp16 number's half step

    def __init__(self, lens, *, kv_heads=2, dim=64, page=16, layout="hnd", dtype=BF, shift=1.0,
                 device="cuda", **kw):
        super().__init__(lens, kv_heads=kv_heads, dim=dim, page=page, layout=layout, dtype=dtype,
                         device=device, **kw)
        self.cache_dtype = U4
        g = torch.Generator(device=device)
        g.manual_seed(99)
        self.c, self.sz, pools = {}, {}, []
        for name, store in (("k", self.k64), ("v", self.v64)):
            pool, sz = pool_u4(self.pages, kv_heads, page, dim, layout, device)
            self.c[name], self.sz[name] = [], []
            for b, x in enumerate(store):
                L = x.shape[0]
                x = x + shift * torch.randn((dim,), generator=g, device=device).double()
                c, w = codes_of(x)
                if L:
                    j = torch.arange(L, device=device)
                    p = torch.tensor(self.owned[b] + [0], device=device)[j // page]
                    pool[p, :, j % page] = packed(c)
                    sz[p, :, j % page] = w
                store[b] = values(c, w)
                self.c[name].append(c)
                self.sz[name].append(w)
            pools.append((pool, sz))
        (k, ks), (v, vs) = pools
        self.cache = sv.KVCache(k, v, ks, vs)

    def reference(self, window=0, scale=None):
        """(out, lse, bound on |error| of out, of lse) in float64."""
        scale = self.D ** -0.5 if scale is None else scale
        outs, lses, tols, ltols = [], [], [], []
        half, tiny = HALF[self.dtype], TINY[self.dtype]
        for b, (n, L) in enumerate(self.lens):
            if n == 0:
                continue
            q = self.q[self.start_list[b]:self.start_list[b + 1]].double().reshape(n, self.H, self.G, self.D)
            k, v, N = self.k64[b], self.v64[b], self.k64[b].shape[0]
            s = torch.einsum("nhgd,lhd->nhgl", q, k) * scale
            at = L - n + torch.arange(n, device=q.device)
            j = torch.arange(N, device=q.device)
            seen = j <= at[:, None]
            if window:
                seen = seen & (j > at[:, None] - window)
            s = s.masked_fill(~seen[:, None, None], -math.inf)
            lse = torch.logsumexp(s, -1) if N else s.new_full(s.shape[:-1], -math.inf)
            p = torch.exp(s - lse[..., None]).nan_to_num(0.0) if N else s
            o = torch.einsum("nhgl,lhd->nhgd", p, v)
            # a score: z sum(q) + s (q.c), sums of head_dim terms in fp32 whose last bit the
            # tensor cores may cut (2^-23 a term), its scaling, and an exponential good to 2 ulp
            ks, vs = self.sz["k"][b].double(), self.sz["v"][b].double()
            if N:
                size = ks[..., 1].abs() + 15 * ks[..., 0]                     # [l, h]
                big = (q.abs().sum(-1)[..., None] * size.T[None, :, None]).masked_fill(
                    ~seen[:, None, None], 0.0).amax(-1) * abs(scale)
                mass = torch.einsum("nhgl,lhd->nhgd", p,
                                    self.c["v"][b].double() * vs[..., :1] + vs[..., 1:].abs())
                # a weight p s enters the product as an fp16 number of 2^9 p s / E, E the largest
                # step rounded up to a power of two: half a step of the smallest, 2^-25, is
                # 2^-34 E, at most 2^-33 of the largest step, times a code of up to 15
                lost = L * 15 * vs[..., 0].amax(0)[None, :, None, None] * 2.0 ** -33
            else:
                big, mass, lost = torch.zeros_like(lse), torch.zeros_like(o), 0.0
            delta = ((self.D + 8) * big + 8) * 2.0 ** -23
            # sums of L terms in fp32 in any order, and of 128 at a time on the tensor cores
            delta = delta + L * 2.0 ** -23
            tol = half * o.abs() + (self.weight + 2 * delta[..., None]) * mass * (1 + half) + lost + tiny
            outs.append(o.reshape(n, -1, self.D))
            lses.append(lse.reshape(n, -1))
            tols.append(tol.reshape(n, -1, self.D))
            ltols.append((2 * delta + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22).reshape(n, -1))
        return torch.cat(outs), torch.cat(lses), torch.cat(tols), torch.cat(ltols)
