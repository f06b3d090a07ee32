"""spec_kv_append_rope: rotated queries and keys against the definition in 64 bits, and what enters
the pages against the definition's fp32 operations, bit for bit."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import Case, E4M3, HALF, TINY, quantise64
from tests._paged_u4 import BF, FP, U4, CaseU4, codes_of, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


def make(lens, cache, **kw):
    if cache == U4:
        return CaseU4(lens, **kw)
    return Case(lens, cache=cache, **kw)


def table_of(positions, rot, base=10000.0):
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def projection(c, heads, seed=1):
    """q, k, v as slices of one wider projection."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn((c.total, heads + 2 * c.H + 1, c.D + 8), generator=g, device="cuda").to(c.dtype)
    w = w[..., :c.D]
    return w[:, :heads], w[:, heads:heads + c.H], w[:, heads + c.H:heads + 2 * c.H]


def rotate(x, angles, interleaved):
    """Rows [total, heads, D] by angles [total, rot], in x's own precision, each operation rounded."""
    rot = angles.shape[1]
    c, s = angles[:, None, :rot // 2].to(x.dtype), angles[:, None, rot // 2:].to(x.dtype)
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def positions_of(c):
    return torch.tensor([L - n + i for n, L in c.lens for i in range(n)], device="cuda")


def check(c, rope, heads=6, interleaved=False, seed=1, **kw):
    q, k, v = projection(c, heads, seed)
    cache = c.cache
    raw = lambda t: t.view(torch.uint8) if t.dtype in (E4M3, U4) else t.view(torch.int16)  # noqa: E731
    before = [(raw(x).clone(), None if s is None else s.clone())
              for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    o = sv.spec_kv_append_rope(cache, k, v, c.table, c.start, c.len, rope, q=q if heads else None,
                               interleaved=interleaved, want_flags=True, **kw)
    torch.cuda.synchronize()
    pos = positions_of(c)
    ok = (pos >= 0) & (pos < rope.shape[0])
    angles = rope[pos.clamp(0, rope.shape[0] - 1)]
    if heads:
        want = rotate(q.double(), angles, interleaved)
        # two products and a sum in fp32, of |x c| + |y s| at most |x| |c| + |y| |s| (1.5 half
        # steps of that), then one rounding
        size = rotate(q.double().abs(), torch.cat([angles[:, :angles.shape[1] // 2].abs(),
                                                   -angles[:, angles.shape[1] // 2:].abs()], 1), interleaved).abs()
        half = angles.shape[1] // 2
        other = rotate(q.double().abs(), torch.cat([angles[:, :half].abs(), angles[:, half:].abs()], 1),
                       interleaved).abs()
        size = torch.maximum(size, other)
        tol = HALF[c.dtype] * want.abs() + size * 2.0 ** -23 + TINY[c.dtype]
        err = (o["q"].double() - want).abs()
        assert bool((err <= tol)[ok].all()), float((err / tol)[ok].max())
        assert not bool(o["q"][~ok].any())
        # and bit for bit as its operations in fp32
        assert torch.equal(o["q"][ok], rotate(q.float(), angles, interleaved).to(c.dtype)[ok])
    rotated = rotate(k.float(), angles, interleaved)
    at = [(c.start_list[b] + i, c.owned[b][(L - n + i) // c.ps], (L - n + i) % c.ps)
          for b, (n, L) in enumerate(c.lens) for i in range(n) if 0 <= L - n + i < rope.shape[0]]
    if at:
        r, p, s = (torch.tensor(z, device="cuda") for z in zip(*at))
        for (want, wants), new in zip(before, (rotated, v.float())):
            if c.cache_dtype == E4M3:
                code, e = quantise64(new)
                want[p, :, s] = code.float().to(E4M3).view(torch.uint8)[r]
                wants[p, :, s] = e[r]
            elif c.cache_dtype == U4:
                code, sz = codes_of(new)
                want[p, :, s] = packed(code)[r]
                wants[p, :, s] = sz[r]
            else:
                want[p, :, s] = new.to(c.dtype)[r].view(torch.int16)
    for (want, wants), x, sc in zip(before, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert torch.equal(raw(x), want)
        if sc is not None:
            a, b = (sc, wants) if sc.dtype == torch.uint8 else (sc.view(torch.int16), wants.view(torch.int16))
            assert torch.equal(a, b)
    return o


KINDS = [(BF, BF), (FP, FP), (BF, E4M3), (FP, E4M3), (BF, U4), (FP, U4)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(32, 32), (32, 16), (64, 64), (96, 32), (96, 48), (128, 128), (128, 112),
                                     (256, 256), (256, 64)])
def test_types_and_sizes(dtype, cache, interleaved, dim, rot):
    c = make([(1, 1), (5, 300), (0, 9), (33, 40), (200, 200)], cache, dim=dim, dtype=dtype, kv_heads=3)
    assert not bool(check(c, table_of(300, rot), interleaved=interleaved)["flags"].any())


@pytest.mark.parametrize("dim,rot", [(16, 16), (80, 32), (80, 80), (112, 96)])
def test_head_sizes_of_16(dim, rot):
    for cache in (BF, E4M3):
        c = make([(5, 300), (33, 40)], cache, dim=dim, kv_heads=3)
        check(c, table_of(300, rot))


@pytest.mark.parametrize("cache", [BF, E4M3, U4])
@pytest.mark.parametrize("page,layout", [(1, "hnd"), (24, "nhd"), (64, "nhd"), (512, "hnd")])
@pytest.mark.parametrize("kv_heads,heads", [(1, 1), (2, 0), (8, 64), (40, 40)])
def test_pages_and_heads(cache, page, layout, kv_heads, heads):
    c = make([(7, 100), (130, 131), (1, 60)], cache, page=page, layout=layout, kv_heads=kv_heads, dim=64)
    assert not bool(check(c, table_of(131, 64), heads=heads)["flags"].any())


@pytest.mark.parametrize("cache", [BF, U4])
def test_many_sequences_and_many_tokens(cache):
    lens = [(b % 5, 3 + (11 * b) % 70 + b % 5) for b in range(500)]
    check(make(lens, cache), table_of(100, 64))
    check(make([(9000, 9001), (1, 4), (801, 801)], cache, kv_heads=1), table_of(9001, 64), heads=3)
    for total in (1, 2, 3, 150, 700, 2433):  # parts of a token's rows to a warp
        check(make([(total, total + 3)], cache, kv_heads=5), table_of(total + 3, 64), heads=15)


def test_far_positions():
    """The angles are the table's: positions near the end of a long one."""
    c = make([(3, 1000000), (2, 500)], BF, page=4096, spare=0)
    check(c, table_of(1000000, 64, base=500000.0))


@pytest.mark.parametrize("cache", [BF, E4M3, U4])
def test_positions_outside_the_table_are_dropped(cache):
    c = make([(6, 40), (4, 2), (3, 38), (2, 41)], cache)
    o = check(c, table_of(38, 64))
    assert o["flags"].tolist() == [sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_LENGTH, 0, sv.FLAG_BAD_LENGTH]
    c = make([(6, 40)], cache)
    q, k, v = projection(c, 6)
    held = c.cache.k.view(torch.uint8).clone()
    o = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, torch.empty((0, 64), device="cuda"),
                               q=q, want_flags=True)
    assert o["flags"].tolist() == [sv.FLAG_BAD_LENGTH] and not bool(o["q"].any())
    assert torch.equal(c.cache.k.view(torch.uint8), held)


@pytest.mark.parametrize("cache", [BF, E4M3, U4])
def test_tokens_without_a_page_still_get_their_queries(cache):
    c = make([(4, 20), (3, 30), (2, 40)], cache)
    rope = table_of(64, 64)
    q, k, v = projection(c, 4)
    want = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)["q"]
    held = c.cache.k.view(torch.uint8).clone()
    c.cache.k.view(torch.uint8).fill_(7)
    c.table[1, 1] = -1
    c.table[2] = 2 ** 31 - 1
    o = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q, want_flags=True)
    assert o["flags"].tolist() == [0, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_PAGE]
    assert torch.equal(o["q"], want)
    got = c.cache.k.view(torch.uint8)
    for page, slots in ((c.owned[0][1], range(4)), (c.owned[1][1], ()), (c.owned[2][2], ())):
        for s in range(c.ps):
            x = got[page, :, s]
            assert torch.equal(x, held[page, :, s]) if s in slots else bool((x == 7).all())


@pytest.mark.parametrize("bad", [(7, 4), (-1, 9), (4, 100)])
def test_rows_that_no_sequence_has_are_left_alone(bad):
    c = make([(4, 20), (3, 30), (2, 40)], U4)
    q, k, v = projection(c, 4)
    rope = table_of(64, 64)
    want = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)["q"]
    start = c.start.clone()
    start[1:3] = torch.tensor(bad)
    out = {"q": torch.full_like(want, 5.0)}
    f = sv.spec_kv_append_rope(c.cache, k, v, c.table, start, c.len, rope, q=q, out=out, want_flags=True)["flags"]
    lens, total = start.tolist(), c.total
    good = [b for b in range(3) if 0 <= lens[b] <= lens[b + 1] <= total]
    assert all((int(f[b]) == 0) == (b in good) or b in good for b in range(3))
    rows = [t for b in good for t in range(lens[b], lens[b + 1])]
    rest = [t for t in range(total) if t not in rows]
    assert bool((out["q"][rest] == 5.0).all())
    # packed rows behind the last sequence
    long = torch.cat([k, k]), torch.cat([v, v]), torch.cat([q, q])
    out = {"q": torch.full((2 * total, *want.shape[1:]), 5.0, dtype=BF, device="cuda")}
    sv.spec_kv_append_rope(c.cache, long[0], long[1], c.table, c.start, c.len, rope, q=long[2], out=out)
    assert torch.equal(out["q"][:total], want) and bool((out["q"][total:] == 5.0).all())


def test_queries_in_place():
    c = make([(4, 20), (3000, 3001)], U4)
    q, k, v = projection(c, 6)
    rope = table_of(3001, 48)
    for interleaved in (False, True):
        want = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q,
                                      interleaved=interleaved)["q"]
        mine = q.contiguous()
        got = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=mine,
                                     interleaved=interleaved, out={"q": mine})["q"]
        assert got is mine and torch.equal(mine, want)


def test_a_rotation_by_nothing_is_an_append():
    for dtype, cache in KINDS:
        c = make([(4, 20), (33, 40)], cache, dtype=dtype)
        q, k, v = projection(c, 6)
        rope = torch.cat([torch.ones(40, 32, device="cuda"), torch.zeros(40, 32, device="cuda")], 1)
        o = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)
        assert torch.equal(o["q"], q)
        held = [t.view(torch.uint8).clone() for t in (c.cache.k, c.cache.v, c.cache.k_scale) if t is not None]
        sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
        now = [t.view(torch.uint8) for t in (c.cache.k, c.cache.v, c.cache.k_scale) if t is not None]
        assert all(torch.equal(a, b) for a, b in zip(held, now))


@pytest.mark.parametrize("cache", [BF, E4M3, U4])
def test_what_is_not_finite_stays_in_its_row(cache):
    """A pair with a NaN or an infinity is not finite; its own row alone holds it (all of it in 4
    bits), and elements that are not rotated stay."""
    c = make([(8, 8)], cache, kv_heads=2, dim=64)
    q, k, v = projection(c, 2)
    rope = table_of(8, 32)
    good = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)["q"].clone()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total)
    k[3, 1, 5], q[2, 0, 7], v[6, 0, 40] = math.inf, math.nan, -math.inf
    o = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)["q"]
    odd = ~torch.isfinite(o)
    assert bool(odd[2, 0, [7, 23]].all()) and int(odd.sum()) == 2
    assert torch.equal(o.masked_fill(odd, 0), good.masked_fill(odd, 0))
    now = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total)
    for name, (t, h, at) in (("k", (3, 1, [5, 21])), ("v", (6, 0, [40]))):
        odd = ~torch.isfinite(now[name])
        assert bool(odd[t, h, at].all())
        assert int(odd.sum()) == (64 if cache == U4 else len(at))
        other = torch.ones(8, 2, dtype=torch.bool, device="cuda")
        other[t, h] = False
        assert torch.equal(now[name][other], held[name][other])


def test_another_stream_and_a_graph():
    c = make([(5, 100), (5, 60)], U4)
    q, k, v = projection(c, 4)
    q = q.contiguous()
    rope = table_of(100, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o = sv.spec_kv_append_rope(c.cache, k, v, c.table, c.start, c.len, rope, q=q)["q"]
    s.synchronize()
    c.len -= 7  # a captured graph follows the lengths
    q.mul_(-3)
    g.replay()
    torch.cuda.synchronize()
    pos = positions_of(c) - 7
    assert torch.equal(o, rotate(q.float(), rope[pos], False).to(BF))
