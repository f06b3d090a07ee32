"""More of the target's side of a round: rotary positions on the way into the cache, and a cache in 4 bits.

A target with rotary positions rotates the queries and keys of a chunk before the keys enter the
paged cache; the cache may hold each token's head vectors as 4-bit codes with a step and a zero of
their own; the chunk attends over that cache; and a prefix may be read back. Three operators:

  append   spec_kv_append_rope   a chunk's queries and keys rotated by position, keys and values
                                 into the pages (16 bits, e4m3, or 4 bits; a 4-bit case reads the
                                 new tokens back in the same pass, as one does who continues on
                                 the values that the cache really holds)
  read     spec_kv_read          tokens out of 4-bit pages
  attend   spec_chunk_attention  a ragged chunk of queries per sequence over 4-bit pages

A 4-bit row of D values: z = bf16(smallest), s = bf16((largest - z) / 15) but 2^-120 at least,
codes c = round((x - z) / s) in 0..15, two to a byte (the even element low); it stands for z + s c.

`run` computes each in plain torch operations in 32 bits, or, where `own` is true, calls the
library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1, "u4": 0.5}
SCALE_BYTES = {"bf16": 0, "fp16": 0, "e4m3": 1, "u4": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(name, op, B, n, ctx, heads, kv_heads, dim, page, dtype, cache="u4", layout="hnd",
          window=0, rot=0, pairs="halves"):
    """B sequences with up to n new tokens each (read: n tokens to read), the longest ctx long with
    them; rot: rotated elements of a head; pairs: (i, i + rot/2) "halves", or (2i, 2i+1) "next"."""
    return {"name": name, "op": op, "B": B, "n": n, "ctx": ctx, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype, "cache": cache, "layout": layout,
            "window": window, "rot": rot, "pairs": pairs}


def listed():
    return [
        # one user, one new token after a short prompt: all latency
        _case("attend one token", "attend", 1, 1, 777, 32, 8, 128, 16, "bf16"),
        # a verification round of gamma = 4 over 64 sequences of mixed length, pages token-major
        _case("attend round of 64", "attend", 64, 5, 8192, 32, 8, 128, 32, "bf16", layout="nhd"),
        # gamma = 8 over long caches, eight query heads to a key head
        _case("attend long round", "attend", 32, 9, 40000, 64, 8, 128, 64, "bf16"),
        # one very long document, gamma = 5, two key heads: the work is split along the keys
        _case("attend one long cache", "attend", 1, 6, 200003, 16, 2, 64, 128, "fp16"),
        # a prompt taken in chunks: up to 4096 new tokens on top of what is cached
        _case("attend prompt chunk", "attend", 2, 4096, 8192, 32, 8, 128, 64, "bf16"),
        # odd everything: groups of 5 heads, 96 wide, a sliding window
        _case("attend window", "attend", 5, 2001, 3501, 20, 4, 96, 16, "fp16", layout="nhd", window=1000),
        # one user's new token, rotated into a 16-bit cache: all latency
        _case("append one token", "append", 1, 1, 777, 32, 8, 128, 16, "bf16", "bf16", rot=128),
        # the cache write of a round of 64 into e4m3
        _case("append round, e4m3", "append", 64, 5, 8192, 32, 8, 128, 32, "bf16", "e4m3", rot=128),
        # a batch of prompts into 4 bits, and back
        _case("append prompts, 4 bits", "append", 8, 16001, 16001, 32, 8, 128, 64, "bf16", rot=128),
        # neighbours as pairs, a third of the head rotated, groups of 5, later chunks of prompts
        _case("append chunks, 4 bits", "append", 5, 2001, 3501, 20, 4, 96, 16, "fp16", layout="nhd", rot=32,
              pairs="next"),
        # a prefix read back: a small one, and a large batch
        _case("read prefix", "read", 1, 600, 600, 0, 8, 64, 16, "fp16", layout="nhd"),
        _case("read prefixes", "read", 16, 16001, 16001, 0, 8, 128, 32, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "read"])
    dim = rng.choice([64, 96, 128])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    layout = rng.choice(["hnd", "nhd"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    more = {}
    if op in ("append", "read"):
        total = _log(rng, 1, 90000)
        B = min(_log(rng, 1, 64), total)
        n = -(-total // B)
        ctx = n + (rng.choice([0, _log(rng, 1, 30000)]) if op == "append" else 0)
        if op == "read":
            group = 0
        else:
            group = min(group, 32 // kv_heads)
            more = {"cache": rng.choice(["u4", "u4", "e4m3", dtype]),
                    "rot": rng.choice([dim, dim, dim // 2, 32]),
                    "pairs": rng.choice(["halves", "halves", "next"])}
    else:
        if rng.random() < 0.6:  # single tokens and verification rounds
            n = rng.choice([1, 1, 2, 4, 5, 6, 9, 17, 33])
            tokens = _log(rng, 64, 600000)
            B = min(_log(rng, 1, 128), max(1, tokens // (n + 16)))
        else:  # stretches of prompts
            n = _log(rng, 40, 4096)
            B = max(1, min(_log(rng, 1, 16), 8192 // n))
            tokens = B * (n + _log(rng, 1, 4096))
            group = min(group, max(1, 32 // kv_heads))
        ctx = max(n, tokens // B)
        more = {"window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}
    c = _case("", op, B, n, ctx, kv_heads * group, kv_heads, dim, page, dtype, layout=layout, **more)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, length with them) of every sequence: ragged, by the case alone."""
    r = random.Random("lengths %d %d %d" % (case["B"], case["n"], case["ctx"]))
    n, kv = [], []
    for b in range(case["B"]):
        # rounds have the same chunk everywhere; prompts differ; the first one is whole
        m = case["n"] if b == 0 or case["n"] <= 64 else r.randint(case["n"] // 4, case["n"])
        if case["op"] == "read" or case["n"] == case["ctx"]:
            L = m
        else:
            L = case["ctx"] if b == 0 else r.randint(max(m, case["ctx"] // 8), max(m, case["ctx"]))
        n.append(m)
        kv.append(L)
    return n, kv


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _pow2(k):
    """2^k in fp32 by its bits, -126 <= k <= 127."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _e4m3(x):
    """e4m3 codes and power-of-two exponents (biased by 127) of fp32 rows [..., dim]: the
    smallest power of two with amax / scale <= 448, at least 2^-120."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax == 0, torch.full_like(k, -120), k).clamp_min(-120)
    return (x * _pow2(-k)[..., None]).to(torch.float8_e4m3fn), (k + 127).to(torch.uint8)


def _u4(x):
    """Packed 4-bit codes [..., dim/2] and (step, zero) bf16 [..., 2] of fp32 rows [..., dim]."""
    z = x.amin(-1).to(torch.bfloat16)
    half = z.float() * 0.5
    s = ((x.amax(-1) * 0.5 - half) * (1.0 / 7.5)).to(torch.bfloat16).clamp_min(2.0 ** -120)
    c = torch.round((x * 0.5 - half[..., None]) / (s.float() * 0.5)[..., None])
    c = c.clamp(0.0, 15.0).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([s, z], -1)


def _u4_values(codes, sz, wide):
    """What packed codes and their (step, zero) stand for, in `wide`."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(wide)
    sz = sz.to(wide)
    return c * sz[..., :1] + sz[..., 1:]


def _pool(case, pages, g):
    """A cache pool [pages, kv_heads, page, dim] (any order in memory) holding earlier tokens."""
    H, ps, D = case["kv_heads"], case["page"], case["dim"]
    hnd = case["layout"] == "hnd"
    shape = (pages, H, ps, D) if hnd else (pages, ps, H, D)
    gain = torch.exp(0.4 * torch.randn((D,), generator=g, device=DEV))  # channels differ in size
    bias = 0.5 * torch.randn((D,), generator=g, device=DEV)             # and are not centred
    x = torch.randn(shape, generator=g, device=DEV) * gain + bias
    if case["cache"] == "u4":
        x, s = _u4(x)
        s = s if hnd else s.transpose(1, 2).contiguous()
    elif case["cache"] == "e4m3":
        x, s = _e4m3(x)
        s = s if hnd else s.transpose(1, 2).contiguous()
    else:
        x, s = x.to(TYPES[case["cache"]]), None
    return (x if hnd else x.transpose(1, 2)), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    B, H, D, ps = case["B"], case["kv_heads"], case["dim"], case["page"]
    n, kv = _lengths(case)
    # an append touches its chunk's pages alone: the pool holds no others
    skip = [(L - m) // ps if case["op"] == "append" else 0 for m, L in zip(n, kv)]
    need = [-(-L // ps) - f for L, f in zip(kv, skip)]
    width = max(a + f for a, f in zip(need, skip))
    pages = sum(need) + 3
    kp, ks = _pool(case, pages, g)
    vp, vs = _pool(case, pages, g)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    # sequence b owns need[b] pages of the shuffled pool; the rest of its row is never read
    first, start = [0], [0]
    for c, m in zip(need, n):
        first.append(first[-1] + c)
        start.append(start[-1] + m)
    at = torch.arange(width, device=DEV)[None] - torch.tensor(skip, device=DEV)[:, None]
    owned = (at >= 0) & (at < torch.tensor(need, device=DEV)[:, None])
    slot = at + torch.tensor(first[:-1], device=DEV)[:, None]
    table = torch.where(owned, order[slot.clamp(0, pages - 1)], -1).to(torch.int32)
    st = {"case": case, "k": kp, "v": vp, "ks": ks, "vs": vs, "table": table,
          "start": torch.tensor(start, dtype=torch.int32, device=DEV),
          "len": torch.tensor(kv, dtype=torch.int32, device=DEV),
          "total": start[-1], "n_max": max(n), "kv_max": max(kv)}
    # the projection's output holds queries, keys and values side by side
    rows = case["heads"] + (2 * H if case["op"] == "append" else 0)
    if rows:
        bias = 0.5 * torch.randn((rows, D), generator=g, device=DEV)
        qkv = torch.randn((start[-1], rows, D), generator=g, device=DEV).add_(bias).to(TYPES[case["dtype"]])
        st["q"] = qkv[:, :case["heads"]]
        if case["op"] == "append":
            st["new_k"], st["new_v"] = qkv[:, case["heads"]:case["heads"] + H], qkv[:, -H:]
            # the model's table of rotations: cosines, then sines, of position times frequency
            f = 10000.0 ** (-2.0 * torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV) / case["rot"])
            a = torch.arange(max(kv), dtype=torch.float64, device=DEV)[:, None] * f
            st["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
    # the first token to read: a whole prefix, or the chunk just written
    firsts = [L - m for m, L in zip(n, kv)] if case["op"] == "append" else [0] * B
    st["first"] = torch.tensor(firsts, dtype=torch.int32, device=DEV)
    if own:  # the handle that a server keeps beside its pool
        import speculative_decoding_verification_21_gb300 as sv
        st["cache"] = sv.KVCache(kp, vp, ks, vs)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"append": _append, "read": _read, "attend": _attend}[st["case"]["op"]](st)


def _run_own(st):
    import speculative_decoding_verification_21_gb300 as sv
    c = st["case"]
    if c["op"] == "append":
        r = sv.spec_kv_append_rope(st["cache"], st["new_k"], st["new_v"], st["table"], st["start"],
                                   st["len"], st["rope"], q=st["q"], interleaved=c["pairs"] == "next")
        return _appended(st, r["q"], lambda: _own_read(sv, st))
    if c["op"] == "read":
        return _own_read(sv, st)
    r = sv.spec_chunk_attention(st["q"], st["cache"], st["table"], st["start"], st["len"],
                                window=c["window"])
    return {"out": r["out"], "lse": r["lse"]}


def _own_read(sv, st):
    r = sv.spec_kv_read(st["cache"], st["table"], st["first"], st["start"], st["total"],
                        dtype=TYPES[st["case"]["dtype"]])
    return {"k": r["k"], "v": r["v"]}


def _appended(st, q, read):
    """An append's outputs: the pools, or for 4 bits the values that the new tokens have there."""
    if st["case"]["cache"] == "u4":
        return {"q": q, **read()}
    r = {"q": q, "k": st["k"], "v": st["v"]}
    if st["ks"] is not None:
        r["ks"], r["vs"] = st["ks"], st["vs"]
    return r


def _rows(st):
    """(sequence, index within its chunk) of every packed row."""
    t = torch.arange(st["total"], device=DEV)
    b = torch.searchsorted(st["start"][1:], t, right=True)
    return b, t - st["start"][b]


def _rotated(x, angles, pairs):
    """fp32 rows [total, heads, dim] with their first elements rotated; angles [total, rot]."""
    rot = angles.shape[1]
    cos, sin = angles[:, None, :rot // 2], angles[:, None, rot // 2:]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if pairs == "halves" else \
        (x[..., 0:rot:2], x[..., 1:rot:2])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.cat(y, -1) if pairs == "halves" else torch.stack(y, -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _append(st):
    c, (b, i) = st["case"], _rows(st)
    pos = st["first"][b] + i
    page, at = st["table"][b, pos // c["page"]].long(), pos % c["page"]
    angles = st["rope"][pos]
    q = _rotated(st["q"].float(), angles, c["pairs"]).to(TYPES[c["dtype"]])
    k = _rotated(st["new_k"].float(), angles, c["pairs"])
    for pool, scale, new in ((st["k"], st["ks"], k), (st["v"], st["vs"], st["new_v"].float())):
        if c["cache"] == "u4":
            pool[page, :, at], scale[page, :, at] = _u4(new)
        elif c["cache"] == "e4m3":
            codes, e = _e4m3(new)
            pool.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = e
        else:
            pool[page, :, at] = new.to(pool.dtype)
    return _appended(st, q, lambda: _read(st))


def _gather(st, page, at, wide):
    """Tokens out of 4-bit pages, [..., kv_heads, dim] in `wide`."""
    return [_u4_values(pool[page, :, at], scale[page, :, at], wide)
            for pool, scale in ((st["k"], st["ks"]), (st["v"], st["vs"]))]


def _read(st):
    b, i = _rows(st)
    pos = st["first"][b] + i
    ps = st["case"]["page"]
    k, v = _gather(st, st["table"][b, pos // ps].long(), pos % ps, torch.float32)
    dt = TYPES[st["case"]["dtype"]]
    return {"k": k.to(dt), "v": v.to(dt)}


def _attend(st):
    c = st["case"]
    B, H, G, D, ps = c["B"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["page"]
    b, i = _rows(st)
    n = st["start"][1:] - st["start"][:-1]
    # queries and keys padded to the longest of the batch
    q = torch.zeros((B, st["n_max"], H, G, D), device=DEV)
    q[b, i] = st["q"].float().reshape(-1, H, G, D)
    j = torch.arange(st["kv_max"], device=DEV)
    page = st["table"][:, j // ps].clamp_min(0).long()
    k, v = _gather(st, page, (j % ps).expand(B, -1), torch.float32)
    held = (j < st["len"][:, None])[..., None, None]
    v = torch.where(held, v, 0.0).permute(0, 2, 1, 3)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * st["n_max"], D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).reshape(B, H, G, st["n_max"], -1)
    s = s * (1.0 / math.sqrt(D))
    pos = (st["len"] - n)[:, None] + torch.arange(st["n_max"], device=DEV)
    seen = j <= pos[..., None]
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(B, H, G * st["n_max"], -1), v).reshape(B, H, G, st["n_max"], D) / l
    lse = (m + l.log())[..., 0]
    out = o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, H * G, D).to(TYPES[c["dtype"]])
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[b, i].reshape(-1, H * G)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    n, kv = _lengths(case)
    H, D, heads = case["kv_heads"], case["dim"], case["heads"]
    held = 2 * H * (D * BYTES[case["cache"]] + SCALE_BYTES[case["cache"]])
    plain = 2 * H * D * BYTES[case["dtype"]]
    if case["op"] == "read":
        return {"bytes": sum(n) * (held + plain), "flops": sum(n) * 2 * H * D * 2}
    if case["op"] == "append":  # (the pages of a chunk are hot when it is read back: values out)
        back = plain if case["cache"] == "u4" else 0
        q = 2 * heads * D * BYTES[case["dtype"]]
        positions = max(kv) if case["n"] > 64 else min(sum(n), max(kv))
        return {"bytes": sum(n) * (held + plain + back + q) + positions * 4 * case["rot"],
                "flops": sum(n) * ((heads + H) * 3 * case["rot"] + 2 * H * D * 4)}
    w = case["window"]
    read, pairs = 0, 0
    for m, L in zip(n, kv):
        first = max(0, L - m + 1 - w) if w else 0
        read += L - first
        if w:  # positions L-m .. L-1 see min(position + 1, w) keys each
            grow = max(0, min(L, w) - (L - m))
            pairs += grow * (L - m) + grow * (grow + 1) // 2 + (m - grow) * w
        else:
            pairs += m * (L - m) + m * (m + 1) // 2
    rows = sum(n) * heads
    return {"bytes": read * held + rows * (2 * D * BYTES[case["dtype"]] + 4),
            "flops": 4 * D * heads * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    n, kv = _lengths(case)
    ps, D, H = case["page"], case["dim"], case["kv_heads"]
    start = st["start"].tolist()

    def held(key, b, lo, hi):  # [hi-lo, H, D] of sequence b
        j = torch.arange(lo, hi, device=DEV)
        page = st["table"][b].long()[j // ps]
        codes, sz = st[key][page, :, j % ps], st[key + "s"][page, :, j % ps].double()
        x = torch.empty((hi - lo, H, D), dtype=torch.float64, device=DEV)
        x[..., 0::2] = (codes % 16).double()
        x[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
        return x * sz[..., :1] + sz[..., 1:]

    def power(k):  # 2^k in 64 bits by its bits
        return ((k.long() + 1023) << 52).view(torch.float64)

    def near(x):  # to the nearest bf16, in 64 bits
        return x.float().to(torch.bfloat16).double()

    def four_bits(x):
        z = near(x.amin(-1, keepdim=True))
        s = near((x.amax(-1, keepdim=True) - z) / 15.0).clamp_min(2.0 ** -120)
        return torch.round((x - z) / s).clamp(0, 15) * s + z

    def eight_bits(x):
        amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -112)
        m, e = torch.frexp(amax / 448.0)
        k = torch.where(m == 0.5, e - 1, e).clamp_min(-120)
        y = x / power(k)
        # to the nearest of the codes: steps of an eighth of the binade, 2^-9 at least
        step = power(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
        return torch.round(y / step) * step  # ties to even

    if case["op"] == "append":
        half = case["rot"] // 2
        i = torch.arange(half, device=DEV)
        at, to = (i, i + half) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)

        def turned(x, pos):  # complex multiplication
            x = x.double()
            t = st["rope"][pos].double()
            y = torch.complex(x[..., at], x[..., to]) * torch.complex(t[:, :half], t[:, half:])[:, None]
            x[..., at], x[..., to] = y.real, y.imag
            return x

        pools = {k: st[k].to(torch.float64) for k in ("k", "v")} if case["cache"] != "u4" else {}
        q, ks, vs = [], [], []
        for b in range(case["B"]):
            rows = slice(start[b], start[b + 1])
            j = torch.arange(kv[b] - n[b], kv[b], device=DEV)
            q.append(turned(st["q"][rows], j))
            k, v = turned(st["new_k"][rows], j), st["new_v"][rows].double()
            if case["cache"] == "u4":
                ks.append(four_bits(k))
                vs.append(four_bits(v))
                continue
            page = st["table"][b].long()[j // ps]
            for key, x in (("k", k), ("v", v)):
                pools[key][page, :, j % ps] = eight_bits(x) if case["cache"] == "e4m3" else x
        if case["cache"] == "u4":
            return {"q": torch.cat(q), "k": torch.cat(ks), "v": torch.cat(vs)}
        r = {"q": torch.cat(q), **pools}
        return {**r, "ks": None, "vs": None} if case["cache"] == "e4m3" else r
    if case["op"] == "read":
        return {p: torch.cat([held(p, b, 0, n[b]) for b in range(case["B"])]) for p in ("k", "v")}
    G = case["heads"] // H
    out, lse = [], []
    for b in range(case["B"]):
        lo = max(0, kv[b] - n[b] + 1 - case["window"]) if case["window"] else 0
        k, v = (held(p, b, lo, kv[b]) for p in ("k", "v"))
        q = st["q"][start[b]:start[b + 1]].double().reshape(n[b], H, G, D)
        o = torch.empty((n[b], H, G, D), dtype=torch.float64, device=DEV)
        z = torch.empty((n[b], H, G), dtype=torch.float64, device=DEV)
        j = torch.arange(lo, kv[b], device=DEV)
        for h in range(H):
            for t in range(0, n[b], 1024):
                e = min(n[b], t + 1024)
                at = kv[b] - n[b] + torch.arange(t, e, device=DEV)
                bad = j > at[:, None]
                if case["window"]:
                    bad = bad | (j <= at[:, None] - case["window"])
                s = (q[t:e, h].reshape(-1, D) @ k[:, h].T).reshape(e - t, G, -1) / D ** 0.5
                s = s.masked_fill(bad[:, None], -math.inf)
                z[t:e, h] = torch.logsumexp(s, -1)
                o[t:e, h] = torch.exp(s - z[t:e, h, :, None]) @ v[:, h]
        out.append(o.reshape(n[b], H * G, D))
        lse.append(z.reshape(n[b], H * G))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
