"""The target's side of a round: what is measured of its cache, its attention and its verification.

A round of speculative decoding runs the target once over a chunk of new tokens of every
sequence (the gamma drafts and the token before them, or a stretch of a prompt): the new keys
and values are written into a paged cache, possibly quantised; the chunk attends over the
cache; the drafts are verified against the target's probabilities; and a prefix of the cache
may be read back (to move it, or to continue elsewhere).  Four operators:

  append   spec_kv_append       new keys and values into the pages, in 16 bits or as e4m3 with
                                one power-of-two scale per token and head
  read     spec_kv_read         tokens of each sequence out of the pages, in 16 bits
  attend   spec_chunk_attention a ragged chunk of queries per sequence over its pages, causal,
                                grouped heads, optionally a sliding window
  verify   spec_verify_probs    the accept test and the draw from given probabilities and given
                                uniforms

`run` computes each in plain torch operations in 32 bits (64 for the running sums of the draw),
or, where `own` is true, calls the library's entry point.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _attend(name, B, n, ctx, heads, kv_heads, dim, page, dtype, cache, layout="hnd", window=0):
    return {"name": name, "op": "attend", "B": B, "n": n, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "cache": cache,
            "layout": layout, "window": window}


def _move(name, op, B, n, kv_heads, dim, page, dtype, cache, layout="hnd"):
    return {"name": name, "op": op, "B": B, "n": n, "ctx": n, "heads": 0, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype, "cache": cache, "layout": layout,
            "window": 0}


def _verify(name, B, gamma, V, dtype):
    return {"name": name, "op": "verify", "B": B, "gamma": gamma, "V": V, "dtype": dtype}


def listed():
    return [
        # one user, one new token after a short prompt: all latency
        _attend("attend one token", 1, 1, 777, 32, 8, 128, 16, "bf16", "bf16"),
        # a verification round of gamma = 4 over 64 sequences of mixed length, pages token-major
        _attend("attend round of 64", 64, 5, 8192, 32, 8, 128, 32, "bf16", "bf16", "nhd"),
        # gamma = 8 over long quantised caches
        _attend("attend round, e4m3", 32, 9, 40000, 64, 8, 128, 64, "bf16", "e4m3"),
        # one very long document, gamma = 5, two key heads: the work is split along the keys
        _attend("attend one long cache", 1, 6, 200003, 16, 2, 64, 128, "fp16", "fp16"),
        # a prompt taken in chunks: up to 4096 new tokens on top of what is cached
        _attend("attend prompt chunk", 2, 4096, 8192, 32, 8, 128, 64, "bf16", "bf16"),
        # odd everything: groups of 5 heads, 96 wide, a sliding window, quantised cache
        _attend("attend window, e4m3", 5, 2001, 3501, 20, 4, 96, 16, "fp16", "e4m3", "nhd", 1000),
        # the cache write of a round of 64 (small) and of a batch of prompts (large)
        _move("append round, e4m3", "append", 64, 5, 8, 128, 32, "bf16", "e4m3"),
        _move("append prompts, e4m3", "append", 8, 16001, 8, 128, 64, "bf16", "e4m3"),
        # a prefix read back: a small one as it is held, a large one out of e4m3
        _move("read prefix", "read", 1, 600, 8, 64, 16, "fp16", "fp16", "nhd"),
        _move("read prefixes, e4m3", "read", 16, 16001, 8, 128, 32, "bf16", "e4m3"),
        # the accept test and the draw: one user, and a large batch
        _verify("verify one row", 1, 4, 32000, "fp32"),
        _verify("verify batch of 256", 256, 8, 152064, "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "read", "verify"])
    if op == "verify":
        B = _log(rng, 1, 200)
        return {"op": op, "B": B, "gamma": rng.randint(1, 8), "V": _log(rng, 1000, 152064),
                "dtype": rng.choice(["fp32", "bf16"])}
    dim = rng.choice([64, 80, 96, 112, 128])
    cache = rng.choice(["same", "e4m3"])
    dtype = rng.choice(["bf16", "fp16"])
    cache = dtype if cache == "same" else cache
    page = rng.choice([8, 16, 32, 64, 128, 256])
    layout = rng.choice(["hnd", "nhd"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if op in ("append", "read"):
        total = _log(rng, 1, 120000)
        B = min(_log(rng, 1, 64), total)
        n = -(-total // B)
        return {"op": op, "B": B, "n": n, "ctx": n, "heads": 0, "kv_heads": kv_heads, "dim": dim,
                "page": page, "dtype": dtype, "cache": cache, "layout": layout, "window": 0}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
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
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    return {"op": op, "B": B, "n": n, "ctx": ctx, "heads": kv_heads * group, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype, "cache": cache, "layout": layout,
            "window": window}


def _lengths(case):
    """(new tokens, cached tokens after them) of every sequence: ragged, by the case alone."""
    r = random.Random("lengths %d %d %d" % (case["B"], case["n"], case["ctx"]))
    n, kv = [], []
    for b in range(case["B"]):
        # rounds have the same chunk everywhere; prompts differ; the first one is whole
        m = case["n"] if b == 0 or case["n"] <= 64 else r.randint(case["n"] // 4, case["n"])
        L = case["ctx"] if b == 0 else r.randint(max(m, case["ctx"] // 8), max(m, case["ctx"]))
        n.append(m)
        kv.append(m if case["op"] != "attend" else L)
    return n, kv


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _quantise(x):
    """e4m3 codes and power-of-two exponents (biased by 127) of fp32 rows [..., dim]: the
    smallest power of two with amax / scale <= 448, at least 2^-120."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax == 0, torch.full_like(k, -120), k).clamp_min(-120)
    codes = (x * _pow2(-k)[..., None]).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _pow2(k):
    """2^k in fp32 by its bits, -126 <= k <= 127."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _pool(case, pages, g):
    """A cache pool [pages, kv_heads, page, dim] (any order in memory) holding earlier tokens."""
    H, ps, D, dt = case["kv_heads"], case["page"], case["dim"], TYPES[case["cache"]]
    hnd = case["layout"] == "hnd"
    shape = (pages, H, ps, D) if hnd else (pages, ps, H, D)
    gain = torch.exp(0.4 * torch.randn((D,), generator=g, device=DEV))  # channels differ
    x = torch.randn(shape, generator=g, device=DEV) * gain
    if case["cache"] == "e4m3":
        x, s = _quantise(x)
        s = (s if hnd else s.transpose(1, 2)).contiguous()
    else:
        x, s = x.to(dt), None
    return (x if hnd else x.transpose(1, 2)), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    B, H, D, ps = case["B"], case["kv_heads"], case["dim"], case["page"]
    n, kv = _lengths(case)
    need = [-(-L // ps) for L in kv]
    width = max(need)
    pages = sum(need) + 3
    kp, ks = _pool(case, pages, g)
    vp, vs = _pool(case, pages, g)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    # sequence b owns need[b] pages of the shuffled pool; the rest of its row is never read
    first = [0]
    for c in need:
        first.append(first[-1] + c)
    slot = torch.arange(width, device=DEV)[None] + torch.tensor(first[:-1], device=DEV)[:, None]
    owned = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(owned, order[slot.clamp_max(pages - 1)], -1).to(torch.int32)
    start = [0]
    for c in n:
        start.append(start[-1] + c)
    st = {"case": case, "k": kp, "v": vp, "ks": ks, "vs": vs, "table": table,
          "start": torch.tensor(start, dtype=torch.int32, device=DEV),
          "len": torch.tensor(kv, dtype=torch.int32, device=DEV),
          "total": start[-1], "n_max": max(n), "kv_max": max(kv)}
    # the projection's output holds queries, keys and values side by side
    rows = case["heads"] + (2 * H if case["op"] == "append" else 0)
    if rows:
        qkv = torch.randn((start[-1], rows, D), generator=g, device=DEV).to(TYPES[case["dtype"]])
        st["q"] = qkv[:, :case["heads"]]
        if case["op"] == "append":
            st["new_k"], st["new_v"] = qkv[:, case["heads"]:case["heads"] + H], qkv[:, -H:]
    if case["op"] == "read":  # whole prefixes: token 0 onwards
        st["first"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:  # the handle that a server keeps beside its pool
        import speculative_decoding_verification_21_gb300 as sv
        st["cache"] = sv.KVCache(kp, vp, ks, vs)
    return st


def _prepare_verify(case, g):
    B, G, V, dt = case["B"], case["gamma"], case["V"], TYPES[case["dtype"]]
    p = torch.empty((B, G + 1, V), dtype=dt, device=DEV)
    q = torch.empty((B, G, V), dtype=dt, device=DEV)
    x = torch.empty((B, G), dtype=torch.int32, device=DEV)
    for b in range(0, B, 32):
        e = min(B, b + 32)
        zt = torch.randn((e - b, G + 1, V), generator=g, device=DEV) * 2.0
        zd = zt[:, :G] + torch.randn((e - b, G, V), generator=g, device=DEV) * 0.4
        p[b:e] = torch.softmax(zt, -1)
        q[b:e] = torch.softmax(zd, -1)
        x[b:e] = torch.multinomial(q[b:e].reshape(-1, V).float(), 1, generator=g).reshape(e - b, G)
    u = torch.rand((B, G + 1), generator=g, device=DEV)
    return {"case": case, "p": p, "q": q, "x": x, "u": u}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"append": _append, "read": _read, "attend": _attend_plain,
            "verify": _verify_plain}[st["case"]["op"]](st)


def _run_own(st):
    import speculative_decoding_verification_21_gb300 as sv
    c = st["case"]
    if c["op"] == "append":
        sv.spec_kv_append(st["cache"], st["new_k"], st["new_v"], st["table"], st["start"], st["len"])
        return _pools(st)
    if c["op"] == "read":
        r = sv.spec_kv_read(st["cache"], st["table"], st["first"], st["start"], st["total"],
                            dtype=TYPES[c["dtype"]])
        return {"k": r["k"], "v": r["v"]}
    if c["op"] == "attend":
        r = sv.spec_chunk_attention(st["q"], st["cache"], st["table"], st["start"], st["len"],
                                    window=c["window"])
        return {"out": r["out"], "lse": r["lse"]}
    r = sv.spec_verify_probs(st["p"], st["q"], st["x"], st["u"])
    return {"tokens": r["tokens"], "counts": r["counts"]}


def _pools(st):
    r = {"k": st["k"], "v": st["v"]}
    if st["ks"] is not None:
        r["ks"], r["vs"] = st["ks"], st["vs"]
    return r


def _rows(st):
    """(sequence, index within its chunk) of every new token."""
    t = torch.arange(st["total"], device=DEV)
    b = torch.searchsorted(st["start"][1:], t, right=True)
    return b, t - st["start"][b]


def _append(st):
    b, i = _rows(st)
    n = st["start"][1:] - st["start"][:-1]
    pos = (st["len"] - n)[b] + i
    page, at = st["table"][b, pos // st["case"]["page"]].long(), pos % st["case"]["page"]
    for pool, scale, new in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
        if scale is not None:
            codes, e = _quantise(new.float())
            pool.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
            scale[page, :, at] = e
        else:
            pool[page, :, at] = new
    return _pools(st)


def _gather(st, page, at, wide):
    """Tokens out of the pages, [..., kv_heads, dim] in `wide`."""
    got = []
    for pool, scale in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        if scale is None:
            got.append(pool[page, :, at].to(wide))
        else:
            x = pool.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).to(wide)
            got.append(x * _pow2(scale[page, :, at].to(torch.int32) - 127)[..., None])
    return got


def _read(st):
    b, i = _rows(st)
    pos = st["first"][b] + i
    ps = st["case"]["page"]
    k, v = _gather(st, st["table"][b, pos // ps].long(), pos % ps, torch.float32)
    dt = TYPES[st["case"]["dtype"]]
    return {"k": k.to(dt), "v": v.to(dt)}


def _attend_plain(st):
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


def _verify_plain(st):
    p, q, x, u = st["p"], st["q"], st["x"].long(), st["u"]
    B, G, V = q.shape
    px = torch.gather(p[:, :G], 2, x[..., None])[..., 0].float()
    qx = torch.gather(q, 2, x[..., None])[..., 0].float()
    ok = (u[:, :G] <= px / qx).to(torch.int32)
    n = torch.cumprod(ok, 1).sum(1)
    row = torch.arange(B, device=DEV)
    pn = p[row, n].float()
    qn = q[row, n.clamp_max(G - 1)].float() * (n < G)[:, None]
    w = (pn - qn).clamp_min(0.0)
    w = torch.where((w > 0).any(1)[:, None], w, pn).double()
    run_sum = torch.cumsum(w, 1)
    # the first entry whose running sum passes u times the total
    t = (run_sum <= u[:, G:].double() * run_sum[:, -1:]).sum(1).clamp_max(V - 1)
    i = torch.arange(G + 1, device=DEV)
    xs = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(i < n[:, None], xs, torch.where(i == n[:, None], t[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "counts": n.to(torch.int32)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "verify":
        B, G, V = case["B"], case["gamma"], case["V"]
        # the row that the token comes from, and the draft's at a rejection: about four rows
        # in five reject somewhere in four drafts of these inputs
        rows = 2.0 - 0.85 ** G
        return {"bytes": B * (rows * V * BYTES[case["dtype"]] + G * 16), "flops": B * rows * V * 2}
    n, kv = _lengths(case)
    H, D = case["kv_heads"], case["dim"]
    held = 2 * H * (D * BYTES[case["cache"]] + (1 if case["cache"] == "e4m3" else 0))
    plain = 2 * H * D * BYTES[case["dtype"]]
    if case["op"] in ("append", "read"):
        return {"bytes": sum(n) * (held + plain), "flops": sum(n) * 2 * H * D * 2}
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
    rows = sum(n) * case["heads"]
    return {"bytes": read * held + rows * (2 * D * BYTES[case["dtype"]] + 4),
            "flops": 4 * D * case["heads"] * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return None  # tokens and counts: whole numbers
    n, kv = _lengths(case)
    ps, D, H = case["page"], case["dim"], case["kv_heads"]
    start = st["start"].tolist()

    def held(pool, scale, b, lo, hi):  # [hi-lo, H, D] of sequence b
        j = torch.arange(lo, hi, device=DEV)
        page = st["table"][b].long()[j // ps]
        x = pool.view(torch.uint8)[page, :, j % ps].view(pool.dtype) if scale is not None \
            else pool[page, :, j % ps]
        x = x.double()
        return x if scale is None else x * power(scale[page, :, j % ps].long() - 127)[..., None]

    def power(k):  # 2^k in 64 bits by its bits
        return ((k.long() + 1023) << 52).view(torch.float64)

    if case["op"] == "append":
        if case["cache"] != "e4m3":
            out = {"k": st["k"].double(), "v": st["v"].double()}
            for b in range(case["B"]):
                j = torch.arange(kv[b] - n[b], kv[b], device=DEV)
                page = st["table"][b].long()[j // ps]
                out["k"][page, :, j % ps] = st["new_k"][start[b]:start[b + 1]].double()
                out["v"][page, :, j % ps] = st["new_v"][start[b]:start[b + 1]].double()
            return out
        out = {"k": st["k"].to(torch.float64), "v": st["v"].to(torch.float64), "ks": None, "vs": None}
        for key in ("k", "v"):
            for b in range(case["B"]):
                j = torch.arange(kv[b] - n[b], kv[b], device=DEV)
                page = st["table"][b].long()[j // ps]
                x = st["new_" + key][start[b]:start[b + 1]].double()
                amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -112)
                m, e = torch.frexp(amax / 448.0)
                k = torch.where(m == 0.5, e - 1, e).clamp_min(-120)
                y = x / power(k)
                # to the nearest of the codes: steps of an eighth of the binade, 2^-9 at least
                step = power(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
                out[key][page, :, j % ps] = torch.round(y / step) * step  # ties to even
        return out
    if case["op"] == "read":
        got = [[held(st[p], st[p + "s"], b, 0, n[b]) for b in range(case["B"])] for p in ("k", "v")]
        return {"k": torch.cat(got[0]), "v": torch.cat(got[1])}
    G = case["heads"] // H
    out, lse = [], []
    for b in range(case["B"]):
        lo = max(0, kv[b] - n[b] + 1 - case["window"]) if case["window"] else 0
        k, v = (held(st[p], st[p + "s"], b, lo, kv[b]) for p in ("k", "v"))
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
