"""spec_chunk_attention over caches of 4-bit codes against the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged_u4 import BF, FP, CaseU4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_types_and_head_sizes(dtype, dim, layout):
    CaseU4([(1, 1), (5, 300), (0, 9), (33, 40), (150, 700)], dim=dim, dtype=dtype, layout=layout).check()


@pytest.mark.parametrize("page", [1, 8, 16, 24, 32, 64, 128, 256])
def test_pages(page):
    CaseU4([(1, 777), (6, 130), (129, 129)], page=page, dim=128, group=3).check()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 27, 40, 64, 80, 100, 128])
def test_groups(group):
    CaseU4([(1, 300), (3, 129), (40, 200)], group=group, dim=64, kv_heads=1).check()


@pytest.mark.parametrize("n", [1, 2, 4, 8, 9, 10, 16, 17, 20, 33, 79, 80, 81, 300])
def test_chunk_lengths(n):
    """Query rows of an item around every tile width."""
    CaseU4([(n, n), (n, n + 1), (n, n + 400)], group=4, dim=128, kv_heads=2).check()


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_lengths_around_tiles(L):
    CaseU4([(1, L), (min(L, 5), L)], dim=128, group=8, kv_heads=1).check()


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 1000, 2 ** 31 - 1])
def test_windows(window):
    CaseU4([(1, 700), (5, 300), (200, 513), (7, 7)], dim=96, group=5).check(window=window)


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e-3, 1.0, -0.125, -1.0])
def test_scales(scale):
    CaseU4([(5, 700), (40, 150), (1, 3)], dim=128).check(scale=scale)


def test_long_caches_cut_over_many_ctas():
    CaseU4([(1, 30011), (5, 20000), (2, 3)], dim=64, kv_heads=2, group=8).check()
    CaseU4([(3, 60000)], dim=128, kv_heads=1, group=5).check()


def test_many_sequences():
    CaseU4([(1 + b % 6, 6 + (37 * b) % 500) for b in range(300)], dim=64, kv_heads=3, group=2).check()


def test_rows_of_very_different_sizes():
    """Steps that differ by 2^16 from token to token."""
    CaseU4([(5, 700), (40, 150)], dim=128, scale_spread=8).check(scale=1e-4)


def test_large_scores():
    """Maxima that rise along the keys: what was summed before is scaled down."""
    c = CaseU4([(4, 1500), (100, 600)], dim=64)
    for b in range(2):
        # keys grow by position, in steps and zeros alike
        L = c.k64[b].shape[0]
        f = 2.0 ** torch.floor(torch.linspace(-4, 3, L, device="cuda")).double()
        c.k64[b] *= f[:, None, None]
        c.sz["k"][b] = (c.sz["k"][b].double() * f[:, None, None]).to(BF)
        j = torch.arange(L, device="cuda")
        p = torch.tensor(c.owned[b], device="cuda")[j // c.ps]
        c.cache.k_scale[p, :, j % c.ps] = c.sz["k"][b]
    c.check(scale=1.0)


def test_constant_rows_and_zero_rows():
    """Steps at their smallest (2^-120) beside ordinary ones."""
    c = CaseU4([(3, 300)], dim=64)
    for t in (0, 5, 130, 299):
        for name, store in (("k", c.k64), ("v", c.v64)):
            scales = c.cache.k_scale if name == "k" else c.cache.v_scale
            pool = c.cache.k if name == "k" else c.cache.v
            page, slot = c.owned[0][t // c.ps], t % c.ps
            z = 0.0 if t % 2 else 1.25
            scales[page, :, slot, 0], scales[page, :, slot, 1] = 2.0 ** -120, z
            pool[page, :, slot] = 0
            c.sz[name][0][t, :, 0], c.sz[name][0][t, :, 1] = 2.0 ** -120, z
            c.c[name][0][t] = 0
            store[0][t] = z
    c.check()


def test_a_query_that_sees_nothing():
    c = CaseU4([(5, 2), (3, 0), (2, 40)])
    o = c.attend()
    torch.cuda.synchronize()
    out, lse = o["out"], o["lse"]
    assert not bool(out[:3].any()) and bool(torch.isneginf(lse[:3]).all())
    assert not bool(out[5:8].any()) and bool(torch.isneginf(lse[5:8]).all())
    assert bool(torch.isfinite(lse[3:5]).all()) and bool(torch.isfinite(lse[8:]).all())
    want, wlse, tol, _ = c.reference()
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_are_not_finite_reach_their_readers_alone(which, dim):
    """A token whose row was not finite (its step and zero are NaN): the queries that see it are NaN
    (of a value row: their outputs alone), the others what they were."""
    c = CaseU4([(40, 200), (6, 300)], dim=dim)
    want = c.attend()
    for pos in (170, 199):
        page, slot = c.owned[0][pos // c.ps], pos % c.ps
        if which != "v":
            c.cache.k_scale[page, 1, slot] = math.nan
        if which != "k":
            c.cache.v_scale[page, 1, slot] = math.nan
    o = c.attend()
    torch.cuda.synchronize()
    G = c.G
    reads = torch.zeros((c.total, 2 * G), dtype=torch.bool, device="cuda")
    reads[10:40, G:] = True  # positions 170 .. 199 of head 1
    assert bool(torch.isnan(o["out"][reads]).all())
    assert torch.equal(o["out"][~reads], want["out"][~reads])
    assert torch.equal(o["lse"][~reads], want["lse"][~reads])
    if which == "v":
        assert torch.equal(o["lse"], want["lse"])
    else:
        assert bool(torch.isnan(o["lse"][reads]).all())


def test_queries_that_are_not_finite():
    for dim in (128, 160):
        c = CaseU4([(12, 200)], dim=dim)
        want = c.attend()
        c.q[3, 2, 5], c.q[4, 1, 0], c.q[5, 0, 1] = math.nan, math.inf, -math.inf
        o = c.attend()
        bad = torch.zeros((12, c.q.shape[1]), dtype=torch.bool, device="cuda")
        bad[3, 2] = bad[4, 1] = bad[5, 0] = True
        assert bool(torch.isnan(o["out"][bad]).all())
        assert torch.equal(o["out"][~bad], want["out"][~bad])
        assert torch.equal(o["lse"][~bad], want["lse"][~bad])


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 30, 2.0 ** 100])
def test_queries_of_any_size(size):
    """bf16 queries far outside fp16's range, with a scale that brings the scores back; one row holds
    values of very different sizes."""
    c = CaseU4([(3, 300), (20, 150)], dim=128)
    c.q.mul_(size)
    c.q[1, 0, ::2] *= 2.0 ** -20
    c.check(scale=0.1 / size)


def test_zero_queries():
    c = CaseU4([(3, 300)], dim=64)
    c.q[:, :3] = 0
    c.check()


def test_bad_pages_and_lengths():
    for dim in (64, 160):
        c = CaseU4([(5, 100), (5, 300), (2, 60)], dim=dim)
        good = c.attend()
        c.table[1, 3] = -7
        page = c.owned[1][3]
        o = c.attend(want_flags=True)
        assert o["flags"].tolist() == [0, sv.FLAG_BAD_PAGE, 0]
        for rows in (slice(0, 5), slice(10, 12)):
            assert torch.equal(o["out"][rows], good["out"][rows])
        # the page reads as zeros
        c.table[1, 3] = page
        for x in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale):
            x[page] = 0
        z = c.attend()
        assert torch.equal(o["out"], z["out"]) and torch.equal(o["lse"], z["lse"])
        c.len[2] = 10 ** 6
        o = c.attend(want_flags=True)
        assert o["flags"][2].item() & sv.FLAG_BAD_LENGTH
        assert torch.equal(o["out"][:10], z["out"][:10])
        c.len[2] = -4
        o = c.attend(want_flags=True)
        assert o["flags"][2].item() & sv.FLAG_BAD_LENGTH
        assert not bool(o["out"][10:].any()) and bool(torch.isneginf(o["lse"][10:]).all())


def test_rows_behind_the_last_sequence_are_left_alone():
    for dim in (64, 160):
        c = CaseU4([(5, 100), (20, 300)], dim=dim)
        want = c.attend()
        q = torch.cat([c.q, c.q])
        out = {"out": torch.full((50, *want["out"].shape[1:]), 3.0, dtype=BF, device="cuda"),
               "lse": torch.full((50, want["lse"].shape[1]), 3.0, device="cuda")}
        sv.spec_chunk_attention(q, c.cache, c.table, c.start, c.len, out=out)
        for name in ("out", "lse"):
            assert torch.equal(out[name][:25], want[name]) and bool((out[name][25:] == 3.0).all())


def test_the_same_bits_every_time():
    c = CaseU4([(5, 9000), (100, 700), (1, 40000)], dim=128, kv_heads=2, group=4)
    a = c.attend()
    for _ in range(5):
        b = c.attend()
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_streams_and_graphs_with_workspaces_of_their_own():
    c = CaseU4([(5, 5000), (30, 60)], dim=128)
    want = c.attend()
    torch.cuda.synchronize()
    need = max(256, sv.attention_workspace_bytes(c.cache, c.q.shape[1]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = []
    for s in streams:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.attend(workspace=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                o = c.attend(workspace=ws)
        made.append((s, g, o, ws))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g, _, _ in made:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, o, _ in made:
        assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    # lengths are read when the graph runs
    c.len[0] -= 100
    want = c.attend()
    torch.cuda.synchronize()
    for _, g, o, _ in made:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["out"], want["out"])


def test_no_rows_and_no_sequences():
    c = CaseU4([(0, 40), (0, 9)])
    o = c.attend(want_flags=True)
    assert o["out"].shape[0] == 0 and o["flags"].tolist() == [0, 0]


def test_offsets_past_31_bits():
    """Pages at the end of a pool of more than 2^31 bytes."""
    pages, H, ps, D = 20000, 4, 512, 128
    k, v = (torch.empty((pages, H, ps, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, H, ps, 2), dtype=BF, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    c = CaseU4([(4, 1000)], kv_heads=H, page=ps, dim=D)
    want = c.attend()
    at = [pages - 1 - i for i in range(c.pages)]
    for big, small in ((k, c.cache.k), (v, c.cache.v), (ks, c.cache.k_scale), (vs, c.cache.v_scale)):
        big[at] = small
    c.cache = sv.KVCache(k, v, ks, vs)
    c.table[0, :2] = pages - 1 - c.table[0, :2]
    o = c.attend()
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])


def test_rotate_attend_read_together():
    """A prompt and a round: rotated, held in 4 bits, attended over and read back, against the model's
    own arithmetic in 64 bits on what the cache reads as."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    H, heads, D, ps = 2, 8, 64, 16
    cache = sv.alloc_kv_cache(40, H, ps, D, dtype=torch.uint8)
    table = torch.randperm(40, generator=g, device="cuda").to(torch.int32).view(2, 20)
    kv = torch.zeros(2, dtype=torch.int32, device="cuda")
    a = torch.arange(320, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(32, device="cuda").double() / 32)
    rope = torch.cat([a.cos(), a.sin()], 1).float()
    for n in ([200, 37], [5, 5], [5, 5]):
        start = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        kv += torch.tensor(n, dtype=torch.int32, device="cuda")
        qkv = torch.randn((sum(n), heads + 2 * H, D), generator=g, device="cuda").to(BF)
        q, k, v = qkv.split([heads, H, H], 1)
        q = sv.spec_kv_append_rope(cache, k, v, table, start, kv, rope, q=q)["q"]
        o = sv.spec_chunk_attention(q, cache, table, start, kv)
        kv -= torch.tensor([m // 5 if m == 5 else 0 for m in n], dtype=torch.int32, device="cuda")
    kv += 1  # (the last round's chunks are still there)
    read_start = torch.cat([kv.new_zeros(1), kv.cumsum(0).to(torch.int32)])
    held = sv.spec_kv_read(cache, table, torch.zeros_like(kv), read_start, int(read_start[-1]))
    for b in range(2):
        kb, vb = (held[x][read_start[b]:read_start[b + 1]].double() for x in ("k", "v"))
        qb = q[start[b]:start[b + 1]].double().view(5, H, heads // H, D)
        s = torch.einsum("nhgd,lhd->nhgl", qb, kb) * D ** -0.5
        L = kb.shape[0]
        seen = torch.arange(L, device="cuda") <= (L - 5 + torch.arange(5, device="cuda"))[:, None]
        p = torch.softmax(s.masked_fill(~seen[:, None, None], -math.inf), -1)
        want = torch.einsum("nhgl,lhd->nhgd", p, vb)
        mass = torch.einsum("nhgl,lhd->nhgd", p, vb.abs())
        # the values that were read are rounded to bf16 (2^-8 of each), which moves a score by
        # 2^-8 sum |q k| scale at most and a weight by twice that
        big = float((torch.einsum("nhgd,lhd->nhgl", qb.abs(), kb.abs()) * D ** -0.5).max())
        tol = mass * (2.0 ** -8 * 3 + 2 * math.expm1(2.0 ** -8 * big)) + 1e-6
        got = o["out"][start[b]:start[b + 1]].double().view_as(want)
        assert bool(((got - want).abs() <= tol).all())
