"""spec_kv_append and spec_kv_read: the pages hold what the definition says, and nothing else moves."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import Case, E4M3, pow2, quantise64

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


def rows(c, seed=1, spread=0):
    """New keys and values as slices of one wider projection."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn((c.total, 2 * c.H + 1, c.D + 8), generator=g, device="cuda")
    if spread:
        w = w * 2.0 ** torch.randint(-spread, spread + 1, (c.total, 2 * c.H + 1, 1), generator=g,
                                     device="cuda")
    w = w.to(c.dtype)
    return w[:, :c.H, :c.D], w[:, c.H:2 * c.H, :c.D]


def raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(torch.int16)


def places(c):
    """(row, page, slot) of every new token that has a place."""
    for b, (n, L) in enumerate(c.lens):
        for i in range(n):
            pos = L - n + i
            if pos >= 0:
                yield c.start_list[b] + i, c.owned[b][pos // c.ps], pos % c.ps


def check_append(c, new_k, new_v):
    cache = c.cache
    before = [(raw(x).clone(), None if s is None else s.clone())
              for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    o = sv.spec_kv_append(cache, new_k, new_v, c.table, c.start, c.len, want_flags=True)
    torch.cuda.synchronize()
    at = list(places(c))
    if at:
        r, p, s = (torch.tensor(z, device="cuda") for z in zip(*at))
        for (want, wants), new in zip(before, (new_k, new_v)):
            if c.cache_dtype == E4M3:
                code, e = quantise64(new)
                want[p, :, s] = code.float().to(E4M3).view(torch.uint8)[r]
                wants[p, :, s] = e[r]
            else:
                want[p, :, s] = new[r].view(torch.int16)
    for (want, wants), x, sc in zip(before, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        got = raw(x)
        if c.cache_dtype == E4M3:  # either sign of NaN will do
            nan = (want & 0x7f) == 0x7f
            assert torch.equal(nan, (got & 0x7f) == 0x7f)
            assert torch.equal(got.masked_fill(nan, 0), want.masked_fill(nan, 0))
            assert torch.equal(sc, wants)
        else:
            assert torch.equal(got, want)
    return o["flags"].tolist()


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4M3), (FP, E4M3)])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
def test_append(dtype, cache, layout, dim):
    c = Case([(1, 1), (5, 300), (0, 9), (33, 40), (200, 200)], dim=dim, dtype=dtype, cache=cache,
             layout=layout, kv_heads=3)
    assert not any(check_append(c, *rows(c)))


@pytest.mark.parametrize("page", [1, 8, 24, 64, 512])
@pytest.mark.parametrize("kv_heads", [1, 2, 8, 40])
def test_append_pages_and_heads(page, kv_heads):
    for cache in (BF, E4M3):
        c = Case([(7, 100), (130, 131)], page=page, kv_heads=kv_heads, dim=64, cache=cache)
        assert not any(check_append(c, *rows(c)))


def test_append_many_sequences():
    lens = [(b % 5, 3 + (11 * b) % 70 + b % 5) for b in range(500)]
    for cache in (BF, E4M3):
        c = Case(lens, cache=cache)
        assert not any(check_append(c, *rows(c)))


def test_scales_over_the_whole_range():
    """Rows from the smallest to the largest size, on and next to the border of 448 2^k, zeros,
    infinities and NaN."""
    for dtype in (BF, FP):
        c = Case([(64, 64)], dim=64, dtype=dtype, cache=E4M3, kv_heads=2)
        k, v = rows(c, spread=5)
        for t, top in enumerate((448.0, 450.0, 446.0, 3.5, 3.515625, 1.75, 1.7578125, 224.0)):
            k[t] = k[t].clamp(-1, 1)
            k[t, :, 3] = top
        k[8] = 0.0
        k[9, 0, 4], k[9, 1, 5] = math.inf, -math.inf
        k[10, 0, 6] = math.nan
        k[11] = math.nan
        k[12] = torch.finfo(dtype).max
        k[13] = torch.finfo(dtype).tiny
        k[14] = torch.finfo(dtype).tiny / 2
        v[3] = -0.0
        v[4, 0] = torch.linspace(-448, 448, 64)
        assert not any(check_append(c, k, v))


def test_append_drops_what_has_no_place_and_says_so():
    c = Case([(4, 2), (3, 30), (2, 40)])
    k, v = rows(c)
    assert check_append(c, k, v) == [sv.FLAG_BAD_LENGTH, 0, 0]  # two tokens before position 0
    for bad in (-1, 10, 2 ** 31 - 1):  # (the pool below has 10 pages)
        c = Case([(4, 20), (3, 30), (2, 40)])
        k, v = rows(c)
        old = c.cache.k.view(torch.int16).clone()
        c.table[1, 1] = bad
        f = sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len, want_flags=True)["flags"]
        assert f.tolist() == [0, sv.FLAG_BAD_PAGE, 0]
        gone = c.owned[1][1]
        assert torch.equal(c.cache.k.view(torch.int16)[gone], old[gone])
    c = Case([(4, 20), (3, 30), (2, 40)])
    k, v = rows(c)
    for bad in (-5, 2 ** 31 - 1):
        c.len[1] = bad
        f = sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len, want_flags=True)["flags"]
        assert f[0] == 0 and f[2] == 0 and f[1].item() & sv.FLAG_BAD_LENGTH
    c.start[1:3] = torch.tensor([7, 4])  # falls: the second sequence is skipped
    f = sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len, want_flags=True)["flags"]
    assert f[1].item() & sv.FLAG_BAD_LENGTH


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4M3), (FP, E4M3)])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dim,page", [(16, 1), (64, 16), (80, 24), (128, 64), (256, 8)])
def test_read(dtype, cache, layout, dim, page):
    c = Case([(0, 100), (0, 1), (0, 333), (0, 0), (0, 64)], dim=dim, dtype=dtype, cache=cache,
             layout=layout, page=page, scale_spread=3 if cache == E4M3 else 0)
    first, count = [3, 0, 0, 0, 63], [97, 1, 333, 0, 1]
    start = [0]
    for n in count:
        start.append(start[-1] + n)
    o = sv.spec_kv_read(c.cache, c.table, torch.tensor(first, dtype=torch.int32, device="cuda"),
                        torch.tensor(start, dtype=torch.int32, device="cuda"), start[-1],
                        dtype=dtype, want_flags=True)
    torch.cuda.synchronize()
    assert not bool(o["flags"].any())
    for name, held in (("k", c.k64), ("v", c.v64)):
        want = torch.cat([held[b][f:f + n] for b, (f, n) in enumerate(zip(first, count))])
        assert torch.equal(o[name].double(), want), name


def test_read_flags_and_zeros():
    c = Case([(0, 40), (0, 40), (0, 40)])
    c.table[1, 1] = -3
    first = torch.tensor([-2, 0, 0], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 4, 36, 40], dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(c.cache, c.table, first, start, 40, want_flags=True)
    assert o["flags"].tolist() == [sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_PAGE, 0]
    assert not bool(o["k"][:2].any()) and not bool(o["k"][4 + 16:36].any())
    assert torch.equal(o["k"][2:4].double(), c.k64[0][:2])
    assert torch.equal(o["v"][36:].double(), c.v64[2][:4])


def test_a_quantised_round_trip_is_within_half_a_code():
    """append then read: off by at most half a step of the code (2^-4 of the value, or half the
    smallest step of the row's scale)."""
    c = Case([(200, 200)], dim=128, dtype=BF, cache=E4M3)
    k, v = rows(c, spread=8)
    sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total)
    for got, new in ((o["k"], k), (o["v"], v)):
        x = new.double()
        step = pow2(quantise64(x)[1].int() - 127)[..., None] * 2.0 ** -9
        assert bool(((got.double() - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, step / 2)).all())


def test_another_stream_and_a_graph():
    c = Case([(5, 100), (5, 60)], cache=E4M3)
    k, v = rows(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    s.synchronize()
    want = raw(c.cache.k).clone()
    c.cache.k.view(torch.uint8).zero_()
    sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    mid = raw(c.cache.k).clone()
    c.cache.k.view(torch.uint8).zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(raw(c.cache.k), mid)
    r, p, sl = (torch.tensor(z, device="cuda") for z in zip(*places(c)))
    assert torch.equal(want[p, :, sl], mid[p, :, sl])


def test_refusals_of_the_binding():
    c = Case([(2, 20)])
    k, v = rows(c)
    with pytest.raises(TypeError):
        sv.spec_kv_append(c.cache, k.float(), v.float(), c.table, c.start, c.len)
    with pytest.raises(ValueError):
        sv.spec_kv_append(c.cache, k, v.contiguous(), c.table, c.start, c.len)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv_append(c.cache, k.half(), v.half(), c.table, c.start, c.len)
    with pytest.raises(TypeError):
        sv.KVCache(c.cache.k.float(), c.cache.v.float())
    with pytest.raises(ValueError):
        sv.KVCache(c.cache.k, c.cache.v.transpose(1, 2))
    e = sv.alloc_kv_cache(4, 2, 16, 64, dtype=E4M3)
    with pytest.raises(ValueError):
        sv.KVCache(e.k, e.v)
    with pytest.raises(ValueError):
        sv.KVCache(e.k, e.v, e.k_scale[:2], e.v_scale[:2])


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("bad", [2 ** 30, -1, -2 ** 31])
@pytest.mark.parametrize("repeat", [1, 120])  # one token a warp, and four
def test_a_bad_start_costs_only_the_sequences_beside_it(cache, bad, repeat):
    B = 70
    c = Case([(repeat * (1 + b % 3), repeat * (1 + b % 3) + b) for b in range(B)], cache=cache)
    k, v = rows(c)
    first = torch.tensor([L - n for n, L in c.lens], dtype=torch.int32, device="cuda")
    sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    want = sv.spec_kv_read(c.cache, c.table, first, c.start, c.total)
    held = raw(c.cache.k).clone(), raw(c.cache.v).clone()
    r, p, s = (torch.tensor(z, device="cuda") for z in zip(*places(c)))
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor([n for n, _ in c.lens])).cuda()
    for at in (0, 1, 33, 69):
        start = c.start.clone()
        start[at] = bad
        skipped = [b for b in (at - 1, at) if b >= 0]
        kept = (owner[:, None] != torch.tensor(skipped, device="cuda")).all(1)
        o = {x: torch.full_like(want[x], math.nan) for x in ("k", "v")}
        f = sv.spec_kv_read(c.cache, c.table, first, start, c.total, out=o, want_flags=True)["flags"]
        assert f.nonzero().flatten().tolist() == skipped
        for x in ("k", "v"):
            assert torch.equal(o[x][kept], want[x][kept])
            assert bool(torch.isnan(o[x][~kept]).all())  # not written
        for pool in (c.cache.k, c.cache.v):
            raw(pool).zero_()
        f = sv.spec_kv_append(c.cache, k, v, c.table, start, c.len, want_flags=True)["flags"]
        assert f.nonzero().flatten().tolist() == skipped
        for pool, all_ in zip((c.cache.k, c.cache.v), held):
            got = raw(pool)[p, :, s]
            assert torch.equal(got[kept], all_[p, :, s][kept]) and not bool(got[~kept].any())
            raw(pool).copy_(all_)


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("length", [33, 34, 36, 40, 2 ** 31 - 1, 0, 2, -1, -2 ** 31])
def test_new_tokens_outside_the_pages_are_dropped_and_others_kept(cache, length):
    """A table of two pages of 16 and chunks of 4: positions below 0 and from 32 on have no place,
    and the tokens that are there already stay."""
    c = Case([(4, 32), (4, 32)], cache=cache)
    c.table = c.table[:, :2].contiguous()
    c.len[0] = length
    k, v = rows(c)
    before = [raw(x).clone() for x in (c.cache.k, c.cache.v)]
    f = sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len, want_flags=True)["flags"]
    assert f.tolist() == [sv.FLAG_BAD_LENGTH, 0]
    at = [(i, length - 4 + i) for i in range(4) if 0 <= length - 4 + i < 32]
    at = [(i, c.owned[0][q // 16], q % 16) for i, q in at]
    at += [(4 + i, c.owned[1][1], 12 + i) for i in range(4)]
    r, p, s = (torch.tensor(z, device="cuda") for z in zip(*at))
    for pool, want, new in zip((c.cache.k, c.cache.v), before, (k, v)):
        if cache == E4M3:
            want[p, :, s] = quantise64(new)[0].float().to(E4M3).view(torch.uint8)[r]
        else:
            want[p, :, s] = new[r].view(torch.int16)
        assert torch.equal(raw(pool), want)


@pytest.mark.parametrize("dtype,last", [(FP, 63456.0), (BF, 247.0 * 2.0 ** 120)])
def test_the_largest_values_of_a_type_round_up_to_infinity(dtype, last):
    """Codes are rounded to nearest: 248 times the scale becomes 256, past the type's range; what
    lies below that border stays finite."""
    top = torch.finfo(dtype).max
    c = Case([(2, 2)], dim=64, dtype=dtype, cache=E4M3)
    k, v = rows(c)
    k[0, 0, 0], k[0, 0, 1], k[0, 1, 0], k[0, 1, 1] = top, last, -top, -last
    sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total, dtype=dtype)["k"]
    scale = 2.0 ** (8 if dtype == FP else 120)
    assert got[0, :, 0].tolist() == [math.inf, -math.inf]
    assert got[0, :, 1].tolist() == [240 * scale, -240 * scale]
    assert bool(torch.isfinite(got[1]).all())
