"""Caches of 4-bit codes: spec_kv_append and spec_kv_read against the definition, bit for bit."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged_u4 import BF, FP, CaseU4, codes_of, packed, unpacked, values

pytestmark = pytest.mark.gpu


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


def places(c, held=None):
    """(row, page, slot) of every new token that has a place."""
    for b, (n, L) in enumerate(c.lens):
        for i in range(n):
            pos = L - n + i
            if pos >= 0:
                yield c.start_list[b] + i, c.owned[b][pos // c.ps], pos % c.ps


def words(sz):
    return sz.view(torch.int16)


def check_append(c, k, v, call=None):
    cache = c.cache
    before = [(x.clone(), s.clone()) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    if call is None:
        o = sv.spec_kv_append(cache, k, v, c.table, c.start, c.len, want_flags=True)
    else:
        o = call()
    torch.cuda.synchronize()
    at = list(places(c))
    if at:
        r, p, s = (torch.tensor(z, device="cuda") for z in zip(*at))
        for (want, wants), new in zip(before, (k, v)):
            code, sz = codes_of(new)
            want[p, :, s] = packed(code)[r]
            wants[p, :, s] = sz[r]
    for (want, wants), x, sz in zip(before, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert torch.equal(x, want)
        nan = torch.isnan(wants)
        assert torch.equal(torch.isnan(sz), nan)
        assert torch.equal(words(sz).masked_fill(nan, 0), words(wants).masked_fill(nan, 0))
    return o["flags"].tolist()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_append(dtype, layout, dim):
    c = CaseU4([(1, 1), (5, 300), (0, 9), (33, 40), (200, 200)], dim=dim, dtype=dtype, layout=layout,
               kv_heads=3)
    assert not any(check_append(c, *rows(c)))


@pytest.mark.parametrize("page", [1, 8, 24, 64, 512])
@pytest.mark.parametrize("kv_heads", [1, 2, 8, 40])
def test_append_pages_and_heads(page, kv_heads):
    c = CaseU4([(7, 100), (130, 131)], page=page, kv_heads=kv_heads)
    assert not any(check_append(c, *rows(c)))


def test_append_many_sequences_and_many_tokens():
    c = CaseU4([(b % 5, 3 + (11 * b) % 70 + b % 5) for b in range(500)])
    assert not any(check_append(c, *rows(c)))
    c = CaseU4([(9000, 9001), (801, 801)], kv_heads=1)  # (four tokens a warp)
    assert not any(check_append(c, *rows(c)))


def test_rows_of_every_size():
    """Rows from the smallest to the largest values, constant ones, on the borders of two codes, far
    from zero; zeros, infinities and NaN."""
    for dtype in (BF, FP):
        top = torch.finfo(dtype).max
        c = CaseU4([(64, 64)], dim=64, dtype=dtype)
        k, v = rows(c, spread=9)
        k[0] = 0.0
        k[1] = -3.0
        k[2] = torch.arange(64, device="cuda") / 4.0          # a quarter of the codes is a tie
        k[3] = 1000.0 + torch.arange(64, device="cuda") % 3   # the zero is rounded
        k[4] = -1000.0 - torch.arange(64, device="cuda") % 7
        k[5] = torch.finfo(dtype).tiny
        k[6] = torch.finfo(dtype).tiny / 4
        k[6, :, 5] = 0.0
        k[7, 0, 4], k[7, 1, 5] = math.inf, -math.inf
        k[8, 0, 6] = math.nan
        k[9] = math.nan
        k[10] = top
        k[11, :, ::2], k[11, :, 1::2] = top, -top             # the span passes the largest float
        k[12] = -0.0
        k[13, :, 0], k[13, :, 1:] = 1e4, 1.0
        k[14] = torch.linspace(-top, top, 64, device="cuda", dtype=torch.float64).to(dtype)
        v[3] = torch.linspace(-448, 448, 64)
        assert not any(check_append(c, k, v))
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total, dtype=dtype)["k"]
        finite = torch.isfinite(k).all(-1)
        assert bool(torch.isnan(got[~finite]).all())          # such a row is NaN throughout
        # rows that reach the end of their type may read as infinities there: the zero and the step
        # are bf16 (row 10 in fp16: 65504 becomes 65536)
        nearly = [t for t in range(64) if t not in (10, 11, 14)]
        assert bool(torch.isfinite(got[nearly][finite[nearly]]).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_codes_are_within_half_a_step(dtype):
    """A code is off by half a step s, and by what the rounding of the zero and of the step leaves:
    2^-8 of the zero, and 2^-8 of the span at its upper end; a read rounds once more."""
    c = CaseU4([(300, 300)], dim=128, dtype=dtype)
    k, v = rows(c, spread=8)
    k = k + 3
    k, v = k.contiguous(), v.contiguous()
    sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(c.cache, c.table, zero, c.start, c.total, dtype=dtype)
    for got, new in ((o["k"], k), (o["v"], v)):
        x, s = new.double(), codes_of(new)[1][..., :1].double()
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        tol = s * (0.5 + 2.0 ** -20) + 2.0 ** -8 * (lo.abs() + hi - lo)
        tol = tol + torch.finfo(dtype).eps / 2 * (x.abs() + tol)
        assert bool(((got.double() - x).abs() <= tol).all())


def test_append_drops_what_has_no_place_and_says_so():
    c = CaseU4([(4, 2), (3, 30), (2, 40)])
    assert check_append(c, *rows(c)) == [sv.FLAG_BAD_LENGTH, 0, 0]  # two tokens before position 0
    for bad in (-1, 10, 2 ** 31 - 1):  # (the pool below has 10 pages)
        c = CaseU4([(4, 20), (3, 30), (2, 40)])
        k, v = rows(c)
        old = c.cache.k.clone()
        c.table[1, 1] = bad
        f = sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len, want_flags=True)["flags"]
        assert f.tolist() == [0, sv.FLAG_BAD_PAGE, 0]
        gone = c.owned[1][1]
        assert torch.equal(c.cache.k[gone], old[gone])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dim,page", [(32, 1), (64, 16), (96, 24), (128, 64), (160, 32), (256, 8)])
def test_read(dtype, layout, dim, page):
    c = CaseU4([(0, 100), (0, 1), (0, 333), (0, 0), (0, 64)], dim=dim, dtype=dtype, layout=layout,
               page=page, scale_spread=3)
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
        assert torch.equal(o[name], want.float().to(dtype)), name  # z + s c in fp32, then the type


def test_read_flags_and_zeros():
    c = CaseU4([(0, 40), (0, 40), (0, 40)])
    c.table[1, 1] = -3
    first = torch.tensor([-2, 0, 0], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 4, 36, 40], dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(c.cache, c.table, first, start, 40, want_flags=True)
    assert o["flags"].tolist() == [sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_PAGE, 0]
    assert o["k"].dtype == BF  # the default
    assert not bool(o["k"][:2].any()) and not bool(o["k"][4 + 16:36].any())
    assert torch.equal(o["k"][2:4], c.k64[0][:2].float().to(BF))
    assert torch.equal(o["v"][36:], c.v64[2][:4].float().to(BF))


def test_padded_tokens_and_pages():
    """Strides larger than a row, a head and a page need: what lies between is left alone."""
    c = CaseU4([(6, 20), (40, 40)], kv_heads=2, dim=64)
    big = torch.full((c.pages, 3, 2, c.ps, 48), 0x5A, dtype=torch.uint8, device="cuda")
    big_v = torch.full_like(big, 0x5A)
    k, v = big[:, 1, :, :, :32], big_v[:, 1, :, :, :32]
    k.copy_(c.cache.k)
    v.copy_(c.cache.v)
    c.cache = sv.KVCache(k, v, c.cache.k_scale, c.cache.v_scale)
    assert not any(check_append(c, *rows(c)))
    for x in (big, big_v):
        assert bool((x[:, 0] == 0x5A).all()) and bool((x[:, 2] == 0x5A).all())
        assert bool((x[:, 1, :, :, 32:] == 0x5A).all())
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 20, 60], dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(c.cache, c.table, zero, start, 60)
    x = c.cache.k[c.owned[1][0]].transpose(0, 1)
    want = values(unpacked(x), c.cache.k_scale[c.owned[1][0]].transpose(0, 1)).float().to(BF)
    assert torch.equal(o["k"][20:20 + c.ps], want)


def test_offsets_past_31_bits():
    """The last pages of a pool of more than 2^31 elements and bytes (head-major, pages of 512)."""
    pages, H, ps, D = 9000, 4, 512, 256
    k, v = (torch.empty((pages, H, ps, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, H, ps, 2), dtype=BF, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    cache = sv.KVCache(k, v, ks, vs)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    new = torch.randn((700, 2 * H, D), generator=g, device="cuda").to(BF)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    n = torch.tensor([700], dtype=torch.int32, device="cuda")
    sv.spec_kv_append(cache, new[:, :H], new[:, H:], table, start, n)
    code, sz = codes_of(new)
    assert torch.equal(k[pages - 1].transpose(0, 1), packed(code)[:512, :H])
    assert torch.equal(v[pages - 2].transpose(0, 1)[:188], packed(code)[512:, H:])
    o = sv.spec_kv_read(cache, table, torch.zeros_like(n), start, 700)
    assert torch.equal(o["k"], values(code, sz)[:, :H].float().to(BF))
    assert torch.equal(o["v"], values(code, sz)[:, H:].float().to(BF))


def test_another_stream_and_a_graph():
    c = CaseU4([(5, 100), (5, 60)])
    k, v = rows(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sv.spec_kv_append(c.cache, k, v, c.table, c.start, c.len)
            o = sv.spec_kv_read(c.cache, c.table, c.len - 5, c.start, c.total)
    s.synchronize()
    k.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o["k"], values(*codes_of(k)).float().to(BF))
    assert torch.equal(o["v"], values(*codes_of(v)).float().to(BF))


def test_alloc():
    e = sv.alloc_kv_cache(4, 2, 16, 64, dtype=torch.uint8)
    assert e.k.shape == (4, 2, 16, 32) and e.head_dim == 64 and e.k_scale.dtype == BF
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    start = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = sv.spec_kv_read(e, table, zero, start, 64)
    assert not bool(o["k"].any()) and not bool(o["v"].any())
