"""Attention over 4-bit codes by the number of an item's rows: both sides of every count at which
another kernel or another variant of one takes over, what few rows do with masks, rows that are
not finite and scores that rise, and waits that run out (one CTA's queries or first scores are
withheld; it gives up after a short limit, the call returns with every sequence flagged, and the
next call gives what a call that never stalled gives)."""
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


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("n", [7, 8, 9, 16, 17, 24, 25, 32, 33, 48, 49, 64, 65])
def test_rows_around_the_variants_bounds(n, dim, window):
    CaseU4([(n, 700), (n, n + 130)], group=1, dim=dim, dtype=FP if n & 1 else BF).check(window=window)


def widened(c, keys):
    """The same with a table of `keys` keys at least: which kernel takes a call goes by that too."""
    more = -(-keys // c.ps) - c.table.shape[1]
    if more > 0:
        c.table = torch.nn.functional.pad(c.table, (0, more), value=2 ** 30)
    return c


@pytest.mark.parametrize("window", [0, 150, 1500])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("n", [7, 16, 25, 33, 49, 65, 81, 200])
def test_rows_in_wide_tables(n, dim, window):
    """Many rows of narrow heads, of few keys in tables of many."""
    widened(CaseU4([(n, 1700 if window > 150 else 700), (n, n + 130)], group=1, dim=dim,
                   dtype=FP if n & 1 else BF), 4000).check(window=window)


@pytest.mark.parametrize("dim", [32, 64, 96])
@pytest.mark.parametrize("group,n", [(3, 40), (5, 20), (8, 12), (16, 7), (40, 2), (80, 1)])
def test_groups_in_wide_tables(group, n, dim):
    widened(CaseU4([(n, 300), (1, 129), (2 * n, 400)], group=group, dim=dim, kv_heads=1), 2000).check()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dim", [64, 96])
def test_rows_that_are_not_finite_in_wide_tables(which, dim):
    c = widened(CaseU4([(40, 200), (6, 300)], dim=dim), 2000)
    want = c.attend()
    for pos in (170, 199):
        page, slot = c.owned[0][pos // c.ps], pos % c.ps
        (c.cache.k_scale if which == "k" else c.cache.v_scale)[page, 1, slot] = math.nan
    o = c.attend()
    reads = torch.zeros((c.total, 2 * c.G), dtype=torch.bool, device="cuda")
    reads[10:40, c.G:] = True
    assert bool(torch.isnan(o["out"][reads]).all())
    assert torch.equal(o["out"][~reads], want["out"][~reads])
    assert torch.equal(o["lse"][~reads], want["lse"][~reads])


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("L", [1, 16, 17, 127, 128, 129, 256, 257, 385, 2000])
def test_single_tokens(dim, L):
    """From one block of a tile to several stages, one tile or two in the last."""
    CaseU4([(1, L), (1, 3)], group=5, dim=dim, page=32, layout="nhd").check()


def test_batches_of_uneven_chunks():
    """Items of the average chunk's rows: longer chunks are several, shorter ones leave rows empty."""
    CaseU4([(1, 300), (0, 20), (13, 500), (1, 1), (2, 2), (7, 130)], group=3, dim=128).check()
    CaseU4([(1, 300), (0, 20), (13, 500), (1, 1), (2, 2), (7, 130)], group=3, dim=96).check(window=10)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_scores_that_rise_and_fall(dim):
    """Keys in order of their scores, upwards for one head and downwards for the other: maxima and
    sums are rescaled at nearly every tile, or never."""
    c = CaseU4([(2, 1500)], group=2, dim=dim)
    c.q[:] = 6.0 * c.q[:1, :1]
    score = torch.einsum("d,lhd->hl", c.q[0, 0].double(), c.k64[0])
    order = torch.stack([score[0].argsort(), score[1].argsort(descending=True)])
    for h in range(2):
        c.k64[0][:, h] = c.k64[0][order[h], h]
        c.c["k"][0][:, h] = c.c["k"][0][order[h], h]
        c.sz["k"][0][:, h] = c.sz["k"][0][order[h], h]
        j = torch.arange(1500, device="cuda")
        p = torch.tensor(c.owned[0], device="cuda")[j // c.ps]
        codes = c.c["k"][0][:, h]
        c.cache.k[p, h, j % c.ps] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        c.cache.k_scale[p, h, j % c.ps] = c.sz["k"][0][:, h]
    c.check()


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("step", [0.0, 2.0 ** -120, 2.0 ** -101])
@pytest.mark.parametrize("n,dim", [(1, 64), (2, 128), (40, 64), (40, 128)])
def test_rows_of_the_smallest_steps_alone(n, dim, step, which):
    """Every row constant, as zeros that were appended are: a step of 2^-120 (or of a pool as it is
    made, 0) is the largest there is."""
    c = CaseU4([(n, 500)], dim=dim, dtype=FP)
    for name, store, pool, sz in (("k", c.k64, c.cache.k, c.cache.k_scale),
                                  ("v", c.v64, c.cache.v, c.cache.v_scale)):
        if which not in (name, "both"):
            continue
        pool.zero_()
        sz[..., 0] = step
        c.sz[name][0][..., 0] = step
        c.c[name][0].zero_()
        store[0][:] = c.sz[name][0][..., 1:].double()
    c.check()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_rows_that_are_not_finite_reach_few_readers_alone(which, dim):
    c = CaseU4([(6, 200), (3, 300)], group=2, dim=dim)
    want = c.attend()
    page, slot = c.owned[0][197 // c.ps], 197 % c.ps
    (c.cache.k_scale if which == "k" else c.cache.v_scale)[page, 1, slot] = math.nan
    o = c.attend()
    reads = torch.zeros((c.total, 4), dtype=torch.bool, device="cuda")
    reads[3:6, 2:] = True  # positions 197 .. 199 of head 1
    assert bool(torch.isnan(o["out"][reads]).all())
    assert torch.equal(o["out"][~reads], want["out"][~reads])
    assert torch.equal(o["lse"][~reads], want["lse"][~reads])
    if which == "v":
        assert torch.equal(o["lse"], want["lse"])
    else:
        assert bool(torch.isnan(o["lse"][reads]).all())


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 30])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_few_queries_of_any_size(dim, size):
    c = CaseU4([(3, 300), (2, 150)], group=2, dim=dim)
    c.q.mul_(size)
    c.q[1, 0, ::2] *= 2.0 ** -20
    c.check(scale=0.1 / size)


@pytest.mark.parametrize("n", [1, 40])
def test_calls_one_behind_another_share_a_workspace(n):
    """A call's kernels start while the last one's end: its records of what was cut are read till then."""
    c = CaseU4([(n, 30000), (1, 500)], dim=128)
    want = c.attend()
    got = [c.attend() for _ in range(60)]
    assert all(torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"]) for o in got)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("n,L,window", [(1, 3, 0), (1, 22, 0), (6, 23, 0), (24, 40, 0), (90, 100, 0),
                                        (2, 224, 0), (200, 400, 0), (1, 2000, 200), (150, 1000, 16)])
def test_few_keys_and_fp16_outputs(n, L, window, dim):
    """Tables of up to 512 keys, or windows: a weight is the sum of two fp16 numbers there, the second the first
    one's rounding error rounded, at most 2^-11 of 2^-11 off."""
    c = CaseU4([(n, L), (1, 9)], group=4, dim=dim, page=32, dtype=FP)
    c.weight = 2.0 ** -22
    c.check(window=window)


@pytest.mark.parametrize("n", [1, 40])
def test_a_wait_that_runs_out_is_flagged_and_the_context_survives(n):
    """A CTA's share is some tiles of an item here, CTA 3's too.  (one token: the queries are
    withheld; 40 tokens by four heads: the first scores)"""
    c = CaseU4([(n, 40000)], dim=128)
    ws = torch.zeros(sv.attention_workspace_bytes(c.cache, 8), dtype=torch.uint8, device="cuda")
    err = ws[160 * 16:160 * 20].view(torch.int32)  # (behind 160 records of 16 bytes)
    want = c.attend(want_flags=True, workspace=ws)
    assert not bool(want["flags"].any()) and not bool(err.any())
    sv.test_attention_stall(3, 1 << 22)
    try:
        stalled = c.attend(want_flags=True, workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.test_attention_stall(-1, 0)
    assert bool((stalled["flags"] & sv.FLAG_TIMEOUT).all())
    e = err.tolist()
    assert e[3] & 1 and e[3] >> 8 and not any(e[:3] + e[4:])
    for _ in range(3):
        again = c.attend(want_flags=True, workspace=ws)
        assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])
        assert not bool(again["flags"].any())
