"""spec_chunk_attention against the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import Case, E4M3

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4M3), (FP, E4M3)])
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 129)], [(5, 5)], [(5, 128), (5, 127), (5, 300)], [(33, 400), (1, 1), (7, 257)],
])
def test_rounds(lens, dtype, cache):
    Case(lens, dtype=dtype, cache=cache).check()


@pytest.mark.parametrize("page", [1, 4, 8, 16, 24, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("cache", [BF, E4M3])
def test_page_sizes(page, cache):
    """Pages that end inside a tile, and tiles that end inside a page."""
    Case([(3, 2 * page + 1), (6, 130), (2, 515)], page=page, cache=cache, dim=128).check()


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 256])
@pytest.mark.parametrize("dtype,cache", [(FP, FP), (BF, E4M3)])
def test_head_sizes(dim, dtype, cache):
    Case([(4, 200), (70, 70)], dim=dim, dtype=dtype, cache=cache, layout="nhd").check()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 31, 71, 128])
@pytest.mark.parametrize("kv_heads", [1, 3])
def test_groups(group, kv_heads):
    """Grouped heads, from one query head per key head to all of them on one."""
    Case([(1, 150), (9, 140), (40, 300)], group=group, kv_heads=kv_heads).check()


@pytest.mark.parametrize("window", [1, 2, 17, 128, 129, 500])
@pytest.mark.parametrize("cache", [BF, E4M3])
def test_windows(window, cache):
    Case([(1, 700), (5, 133), (90, 400), (200, 200)], cache=cache, dim=128).check(window=window)


def test_prompts():
    """Chunks of many tiles, whole prompts and stretches of them, packed."""
    Case([(300, 300), (129, 1000), (1, 17), (513, 700)], dim=128, group=4).check()
    Case([(257, 257), (64, 2000)], dim=64, group=7, dtype=FP).check(window=300)
    Case([(200, 900), (3, 3)], dim=128, group=8, cache=E4M3).check()


def test_long_cache_is_split_and_joined():
    for cache in (FP, E4M3):
        Case([(6, 50001)], kv_heads=1, group=8, dim=64, page=128, dtype=FP, cache=cache).check()
    Case([(1, 9000), (1, 1), (1, 20000), (1, 3)], kv_heads=2, group=8, dim=128).check()


def test_empty_sequences_and_rows_without_keys():
    """No new tokens, no cached ones, and a chunk longer than its sequence: the rows before
    position 0 see nothing."""
    Case([(0, 40), (3, 3), (0, 0), (5, 2), (2, 0), (1, 77)]).check()
    Case([(300, 100), (4, 0)], dim=128).check()
    Case([(0, 10), (0, 0)]).attend()  # nothing to do


def test_scales():
    for scale in (0.0, 1.0, -0.3, 3.0):
        Case([(5, 300), (60, 200)], dim=64).check(scale=scale)


def test_many_sequences():
    lens = [(1 + b % 4, 1 + (37 * b) % 400 + b % 4) for b in range(700)]
    Case(lens, kv_heads=2, group=2).check()


def test_wide_range_of_token_scales():
    """Keys and values whose sizes differ by 2^12 from token to token."""
    Case([(5, 700), (40, 150)], dim=128, cache=E4M3, scale_spread=6).check(scale=1e-3)


def test_sharp_rows():
    """Scores far apart: the running maximum rises by hundreds along the keys, and falls."""
    for sign in (1.0, -1.0):
        c = Case([(4, 1500), (130, 600)], dim=64, group=4)
        for b, (n, L) in enumerate(c.lens):
            ramp = sign * torch.linspace(-6, 6, L, device="cuda")[:, None, None]
            k = (c.k64[b] * 0.1 + ramp).to(BF)
            j = torch.arange(L, device="cuda")
            p = torch.tensor(c.owned[b], device="cuda")[j // c.ps]
            c.cache.k[p, :, j % c.ps] = k
            c.k64[b] = k.double()
        c.q.abs_()
        c.check()


def test_equal_scores_give_the_mean():
    c = Case([(1, 1000)], dim=64)
    c.q.zero_()
    o = c.check()
    assert torch.allclose(o["lse"], torch.full_like(o["lse"], math.log(1000.0)), atol=1e-6)


def test_infinite_and_nan_values_reach_only_who_sees_them():
    """A NaN and an infinity in the first tokens reach every query; the other sequence, the other
    head and whoever's window is past them keep theirs."""
    c = Case([(3, 400), (3, 400)], dim=64)
    page, slot = c.owned[0][0], 2
    c.cache.v[page, 0, slot, 5] = math.inf
    c.cache.v[page, 0, slot, 6] = math.nan
    clean = Case([(3, 400), (3, 400)], dim=64).attend()["out"]
    o = c.attend()["out"]
    assert bool(torch.isposinf(o[:3, :4, 5]).all()) and bool(torch.isnan(o[:3, :4, 6]).all())
    assert torch.equal(o[3:], clean[3:]) and torch.equal(o[:, 4:], clean[:, 4:])
    assert torch.equal(o[:3, :4, 7:], clean[:3, :4, 7:])
    w = c.attend(window=200)["out"]
    assert bool(torch.isfinite(w).all())


def test_a_nan_key_reaches_its_sequence_and_head_only():
    c = Case([(3, 400), (3, 300)], dim=64)
    clean = c.attend()["out"].clone()
    c.cache.k[c.owned[0][3], 1, 4, 9] = math.nan
    o = c.attend()["out"]
    assert bool(torch.isnan(o[:3, 4:]).all())
    assert torch.equal(o[3:], clean[3:]) and torch.equal(o[:3, :4], clean[:3, :4])


def test_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32 (a pool of 6 GB a side)."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    Case([(5, 600), (2, 100)], kv_heads=2, dim=128, page=64, first_page=180000).check()


def test_bad_pages_are_flagged_and_harm_nobody_else():
    c = Case([(5, 300), (5, 300), (2, 40)], dim=64)
    good = c.attend()["out"].clone()
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        c.table[1, 7] = bad
        o = c.attend(want_flags=True)
        assert o["flags"].tolist() == [0, sv.FLAG_BAD_PAGE, 0]
        assert torch.equal(o["out"][:5], good[:5]) and torch.equal(o["out"][10:], good[10:])


def test_bad_lengths_are_flagged_and_harm_nobody_else():
    c = Case([(5, 300), (5, 300), (2, 40)], dim=64)
    good = c.attend()["out"].clone()
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        c.len[1] = bad
        o = c.attend(want_flags=True)
        assert o["flags"][0] == 0 and o["flags"][2] == 0
        assert o["flags"][1].item() & sv.FLAG_BAD_LENGTH
        assert torch.equal(o["out"][:5], good[:5]) and torch.equal(o["out"][10:], good[10:])
    c.len[1] = 300
    c.start[3] = 1000  # past the packed rows: the last sequence is skipped
    o = c.attend(want_flags=True)
    assert o["flags"].tolist() == [0, 0, sv.FLAG_BAD_LENGTH]
    assert torch.equal(o["out"][:10], good[:10])


def test_same_bits_every_time_and_on_another_stream():
    c = Case([(5, 3000), (300, 700), (1, 9000)], dim=128, group=4)
    a = c.attend()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = c.attend()
    s.synchronize()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_captured_into_a_graph_with_lengths_that_change():
    c = Case([(5, 3000), (5, 700)], dim=128, group=4)
    ws = torch.empty(max(256, sv.attention_workspace_bytes(c.cache, 8)), dtype=torch.uint8,
                     device="cuda")
    out = c.attend(workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.attend(workspace=ws, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.attend(workspace=ws, out=out)
    for L in (3000, 129, 2047, 5):
        c.len[0] = L
        want = c.attend()
        out["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])


def test_refusals_of_the_binding():
    c = Case([(2, 20)])
    with pytest.raises(TypeError):
        sv.spec_chunk_attention(c.q.float(), c.cache, c.table, c.start, c.len)
    with pytest.raises(sv.SpecVerifyError):  # fp16 queries on a bf16 cache
        sv.spec_chunk_attention(c.q.half(), c.cache, c.table, c.start, c.len)
    with pytest.raises(ValueError):
        sv.spec_chunk_attention(c.q[..., :32], c.cache, c.table, c.start, c.len)
    with pytest.raises(ValueError):
        sv.spec_chunk_attention(c.q, c.cache, c.table, c.start[:-1], c.len)
    with pytest.raises(TypeError):
        sv.spec_chunk_attention(c.q, c.cache, c.table.long(), c.start, c.len)
    with pytest.raises(sv.SpecVerifyError):  # 7 query heads on 2 key heads
        sv.spec_chunk_attention(c.q[:, :7], c.cache, c.table, c.start, c.len)


@pytest.mark.parametrize("page", [4, 16, 128])
@pytest.mark.parametrize("cache", [BF, E4M3])
def test_a_nan_key_of_a_later_token_stays_away(page, cache):
    """The last token's key is NaN: the chunk's earlier queries keep their bits."""
    c = Case([(6, 300), (200, 260)], dim=64, page=page, cache=cache)
    clean = c.attend()["out"].clone()
    for b, (n, L) in enumerate(c.lens):
        at = (c.owned[b][(L - 1) // page], slice(None), (L - 1) % page)
        if cache == E4M3:
            c.cache.k.view(torch.uint8)[at] = 0x7f
        else:
            c.cache.k[at] = math.nan
    o = c.attend()["out"]
    for b, (n, L) in enumerate(c.lens):
        last = c.start_list[b + 1] - 1
        assert torch.equal(o[c.start_list[b]:last], clean[c.start_list[b]:last])
        assert bool(torch.isnan(o[last]).all())


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("page", [4, 16, 128])
def test_what_lies_in_front_of_the_window_is_not_read(page, cache):
    """Pages that were given back (their table entries are wild), and NaN in the slots in front
    of the first one seen."""
    c = Case([(5, 700), (40, 333)], dim=64, page=page, cache=cache)
    window = 100
    clean = c.attend(window=window)["out"].clone()
    for b, (n, L) in enumerate(c.lens):
        lo = L - n + 1 - window
        first = lo // page
        for s in range(lo % page):
            at = (c.owned[b][first], slice(None), s)
            for pool, scale in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)):
                if cache == E4M3:
                    pool.view(torch.uint8)[at] = 0xff
                    scale[at] = 255
                else:
                    pool[at] = math.nan
        c.table[b, :first] = 2 ** 31 - 1
    o = c.attend(window=window, want_flags=True)
    assert torch.equal(o["out"], clean) and not bool(o["flags"].any())


@pytest.mark.parametrize("lens", [[(1, 40)], [(5, 3000), (70, 200)]])
def test_outputs_and_queries_on_16_byte_boundaries(lens):
    c = Case(lens, dim=128, group=4)
    want = c.attend()["out"]
    room = torch.zeros(c.total * 8 * 128 + 8, dtype=BF, device="cuda")
    out = room[8:].view(c.total, 8, 128)
    qs = torch.zeros(c.total * 8 * 128 + 8, dtype=BF, device="cuda")[8:].view(c.total, 8, 128)
    qs.copy_(c.q)
    sv.spec_chunk_attention(qs, c.cache, c.table, c.start, c.len, out={"out": out})
    assert torch.equal(out, want) and not bool(room[:8].any())


def test_queries_shared_by_all_tokens():
    """A query tensor expanded along the tokens (stride 0)."""
    c = Case([(7, 90), (3, 200)], dim=64)
    one = c.q[:1].contiguous().expand(c.total, -1, -1)
    # (two kernels: each off by 2^-8 of the value and of the weights' mass on |v| < 6)
    a = sv.spec_chunk_attention(one, c.cache, c.table, c.start, c.len)["out"]
    b = sv.spec_chunk_attention(one.contiguous(), c.cache, c.table, c.start, c.len)["out"]
    assert bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * (6 + b.double().abs())).all())


@pytest.mark.parametrize("cache", [BF, FP, E4M3])
@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("lens,dim,group,window", [
    ([(6, 300), (200, 260), (1, 9)], 64, 4, 0),           # all items cut
    ([(6, 30001)], 64, 8, 0),                             # few rows of many parts
    ([(9, 9), (0, 5), (7, 3)], 80, 1, 0),                 # rows that see nothing
    ([(1500, 1700), (3, 40)], 128, 4, 0),                 # items of two row tiles
    ([(1500, 1700), (130, 500)], 96, 2, 150),
    ([(2 + b % 4, 6 + (37 * b) % 400) for b in range(400)], 128, 2, 0),  # whole items
    ([(2 + b % 4, 6 + (37 * b) % 400) for b in range(400)], 64, 7, 50),
])
def test_values_that_are_not_finite_reach_only_queries_that_see_them(cache, page, lens, dim, group,
                                                                     window):
    """The value of every chunk's last but one token is infinite in one column and NaN in another,
    and with a window so is that of the token 3 places before the chunk: the queries that see
    neither keep within the bounds everywhere, the others in the other columns."""
    dtype = FP if cache == FP else BF
    c = Case(lens, kv_heads=2, dim=dim, group=group, page=page, dtype=dtype, cache=cache)
    out, lse, tol, ltol = c.reference(window)  # (of the finite cache)
    sees = torch.zeros(c.total, dtype=torch.bool)
    for b, (n, L) in enumerate(c.lens):
        for j in (L - 2, L - n - 3 if window else -1):
            if j < 0:
                continue
            at = (c.owned[b][j // page], slice(None), j % page)
            if cache == E4M3:  # (the code has no infinity)
                c.cache.v.view(torch.uint8)[at + (slice(5, 7),)] = 0x7f
            else:
                c.cache.v[at + (5,)] = math.inf
                c.cache.v[at + (6,)] = math.nan
            pos = L - n + torch.arange(n)
            seen = (j <= pos) & ((j > pos - window) if window else True)
            sees[c.start_list[b]:c.start_list[b + 1]] |= seen
    sees = sees.cuda()
    o = c.attend(window=window, want_flags=True)
    ok = (o["out"].double() - out).abs() <= tol
    assert bool(ok[~sees].all())
    assert bool(ok[:, :, :5].all()) and bool(ok[:, :, 7:].all())
    assert not bool(torch.isfinite(o["out"][sees][:, :, 5:7]).any())
    near = (o["lse"] == lse) | ((o["lse"].double() - lse).abs() <= ltol)  # (-inf: nothing seen)
    assert bool(near.all()) and not bool(o["flags"].any())


def test_an_infinite_later_value_inside_a_graph():
    """A captured call mends rows as the eager one does, and only while there is something to."""
    c = Case([(6, 300), (300, 700)], dim=128)
    clean = c.attend()["out"].clone()
    out = {"out": torch.empty_like(clean)}
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.attend(out=out)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            c.attend(out=out)
    at = (c.owned[1][(700 - 1) // c.ps], slice(None), (700 - 1) % c.ps)
    kept = c.cache.v[at].clone()
    for value in (math.inf, math.nan):
        c.cache.v[at] = value
        g.replay()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(out["out"][:-1]).all())
        assert not bool(torch.isfinite(out["out"][-1]).any())
        assert torch.equal(out["out"][:6], clean[:6])
    c.cache.v[at] = kept
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], clean)


def test_queued_on_a_stream_that_is_not_the_current_one():
    """The first call on a stream, and one that needs a larger workspace there, with cut items."""
    s = torch.cuda.Stream()
    for dim in (64, 128):
        c = Case([(5, 3000), (300, 700), (1, 9000)], dim=dim)
        want = c.attend()
        s.wait_stream(torch.cuda.current_stream())
        got = c.attend(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_a_graph_keeps_its_workspace_when_a_later_call_needs_a_larger_one():
    """Captured without workspace=; then heads of 128 on the same stream, and memory taken anew."""
    c = Case([(5, 3000), (300, 700)], dim=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = c.attend()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.attend(out=out)
        wide = Case([(5, 3000), (300, 700)], dim=128)
        wide.attend()
        taken = [torch.full((1 << 22,), math.nan, device="cuda") for _ in range(8)]
        want = c.attend()
        out["out"].zero_()
        g.replay()
        s.synchronize()
    assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])
    assert all(bool(torch.isnan(t).all()) for t in taken)  # the replay wrote to nobody's memory


@pytest.mark.parametrize("window", [50, 2 ** 31 - 1])
@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("page", [4, 16])
def test_windows_over_chunks_longer_than_their_cache(window, cache, page):
    """Rows in front of token 0 beside rows that see keys; the largest window hides nothing."""
    Case([(300, 100), (5, 2), (4, 0), (200, 150)], dim=128, cache=cache, page=page).check(
        window=window)


@pytest.mark.parametrize("page", [4, 16])
def test_a_scale_of_zero_with_large_scores(page):
    """Products of 2^106 times zero: every weight is the same."""
    c = Case([(5, 300), (60, 200)], page=page)
    c.q.mul_(2.0 ** 50)
    c.cache.k.mul_(2.0 ** 50)
    c.k64 = [k * 2.0 ** 50 for k in c.k64]
    c.check(scale=0.0)


@pytest.mark.parametrize("bad", [2 ** 30, -1, -2 ** 31])
@pytest.mark.parametrize("page", [4, 16])
def test_a_bad_start_costs_only_the_sequences_beside_it(page, bad):
    B = 70
    c = Case([(1 + b % 3, 20 + b) for b in range(B)], page=page)
    want = c.attend()
    for at in (0, 1, 33, 69):
        start = c.start.clone()
        start[at] = bad
        o = sv.spec_chunk_attention(c.q, c.cache, c.table, start, c.len, want_flags=True)
        skipped = [b for b in (at - 1, at) if b >= 0]
        assert o["flags"].nonzero().flatten().tolist() == skipped
        for b in range(B):
            if b not in skipped:
                r = slice(c.start_list[b], c.start_list[b + 1])
                assert torch.equal(o["out"][r], want["out"][r]), (at, b)
                assert torch.equal(o["lse"][r], want["lse"][r]), (at, b)


def test_a_bad_start_beside_an_infinite_value():
    """Rows are mended by what they see there too."""
    lens = [(2 + b % 4, 6 + (37 * b) % 400) for b in range(200)]
    c = Case(lens, group=2, dim=128)
    c.start[77] = 2 ** 30
    clean = {k: v.clone() for k, v in c.attend().items()}
    for b, (n, L) in enumerate(lens):  # what the last token alone sees
        c.cache.v[c.owned[b][(L - 1) // c.ps], :, (L - 1) % c.ps, 5] = math.inf
    o = c.attend()
    for b in range(200):
        if b not in (76, 77):
            r = slice(c.start_list[b], c.start_list[b + 1] - 1)
            # (mended: fp32 weights instead of rounded ones)
            d = (o["out"][r].double() - clean["out"][r].double()).abs()
            assert bool((d <= 2.0 ** -7 * (6 + clean["out"][r].double().abs())).all()), b
            assert bool(torch.isposinf(o["out"][c.start_list[b + 1] - 1, :, 5]).all()), b


def best_ms(call):
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("want_lse", [True, False])
@pytest.mark.parametrize("cache", [FP, E4M3])
def test_a_row_that_is_rightly_nan_delays_nobody(cache, want_lse):
    """One NaN in a query, one in a key that a whole sequence sees: no row is computed again (that
    took hundreds of times the call's time)."""
    lens = [(6, 100001), (300, 900), (1, 40)]
    c = Case(lens, kv_heads=1, group=8, dim=64, page=128, dtype=FP, cache=cache)
    clean = {k: v.clone() for k, v in c.attend(want_lse=want_lse).items()}
    ms = best_ms(lambda: c.attend(want_lse=want_lse))
    c.q[2, 3, 5] = math.nan
    page = c.owned[1][0]
    if cache == E4M3:
        c.cache.k.view(torch.uint8)[page, :, 7, 9] = 0x7f
    else:
        c.cache.k[page, :, 7, 9] = math.nan
    o = c.attend(want_lse=want_lse)
    nan = torch.zeros((c.total, 8), dtype=torch.bool, device="cuda")
    nan[2, 3] = True
    nan[6:306] = True
    assert bool(torch.isnan(o["out"][nan]).all())
    assert torch.equal(o["out"][~nan], clean["out"][~nan])
    if want_lse:
        assert bool(torch.isnan(o["lse"][nan]).all())
        assert torch.equal(o["lse"][~nan], clean["lse"][~nan])
    assert best_ms(lambda: c.attend(want_lse=want_lse)) < 10 * ms + 0.2


@pytest.mark.parametrize("want_lse", [True, False])
def test_rows_that_are_rightly_nan_beside_rows_to_mend(want_lse):
    c = Case([(6, 300), (200, 260), (40, 40)], dim=128)
    out, _, tol, _ = c.reference()  # (of the finite cache)
    c.q[3, 2, 1] = math.nan
    for b, (n, L) in enumerate(c.lens):
        c.cache.v[c.owned[b][(L - 1) // c.ps], :, (L - 1) % c.ps] = math.nan
    o = c.attend(want_lse=want_lse)["out"]
    last = torch.zeros(c.total, dtype=torch.bool, device="cuda")
    last[[s - 1 for s in c.start_list[1:]]] = True
    nan = last[:, None].expand(-1, 8).clone()
    nan[3, 2] = True
    assert bool(torch.isnan(o[nan]).all())
    assert bool(((o.double() - out).abs() <= tol)[~nan].all())
