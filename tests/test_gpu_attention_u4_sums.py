"""What sums over 4-bit values lose: codes are centred before they are multiplied, so neither the
sums' last bits nor the weights' roundings grow with values that cancel."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import HALF, TINY
from tests._paged_u4 import BF, FP, CaseU4, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,group,dim", [(1, 4, 128), (5, 4, 64), (6, 8, 64), (9, 8, 128), (9, 8, 64)])
def test_long_sums_that_cancel(n, group, dim, dtype):
    """Values 7 and -8 that add up to nothing, along caches as long as a CTA's share of the work.

    Every 128th key scores higher than the others and holds zeros; the rest have one weight w, an
    fp16 number of 11 bits.  Sums of w (c - 8) stay within 16 w all along, so they are exact in
    24 bits; sums of w c would pass 2^28 of w's last bit.  What is left: w itself, 2^-11 off, in
    each of the (at most four) parts of a cut item, the rounding of 1 / l, l's own sum, and the
    output's."""
    B, H, L, ps = 20, 8, 20000, 32
    pages = L // ps
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    j = torch.arange(L, device="cuda")
    high = j % 128 == 0
    count = torch.cumsum(~high, 0) - 1
    d = torch.arange(dim, device="cuda")
    c = torch.where((8 * (count[:, None] + d)) % 15 < 8, 15, 0).masked_fill(high[:, None], 8).to(torch.uint8)
    k, v = (torch.empty((pages, H, ps, dim // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, H, ps, 2), dtype=BF, device="cuda") for _ in range(2))
    v[:] = packed(c).view(pages, 1, ps, dim // 2)
    vs[..., 0], vs[..., 1] = 1.0, -8.0
    k[:] = torch.randint(0, 256, (dim // 2,), generator=g, device="cuda").to(torch.uint8)
    ks[..., 0] = 0.25
    ks[..., 1] = torch.where(high, -1.96875, -2.0).to(BF).view(pages, 1, ps)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.empty_like(table)
    at[table.long()] = torch.arange(pages, device="cuda", dtype=torch.int32)
    for x in (k, v, ks, vs):  # page table[i] holds the i-th tokens
        x.copy_(x[at.long()])
    q = torch.ones((B * n, H * group, dim), device="cuda", dtype=dtype)
    start = n * torch.arange(B + 1, device="cuda", dtype=torch.int32)
    kv = torch.full((B,), L, device="cuda", dtype=torch.int32)
    o = sv.spec_chunk_attention(q, sv.KVCache(k, v, ks, vs), table.repeat(B, 1), start, kv)["out"]
    # the scores differ by dim^1/2 / 32
    w = torch.exp(torch.where(high, 0.0, -dim ** 0.5 / 32).double())
    top = torch.cumsum(w[:, None] * (c.double() - 8), 0)[L - n:]
    low = torch.cumsum(w, 0)[L - n:, None]
    want = (top / low).repeat(B, 1)[:, None]
    tol = HALF[dtype] * want.abs() + 4 * 2.0 ** -11 * 16 / low.repeat(B, 1)[:, None] + L * 2.0 ** -23 * want.abs()
    assert bool(((o.double() - want).abs() <= tol + TINY[dtype]).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160])
def test_values_in_the_middle_of_their_range(dim, window, dtype):
    """Code 8 of steps s and zeros -8 s: every value is zero, and so is every output, whatever the
    weights were rounded to."""
    c = CaseU4([(1, 3), (6, 900), (90, 1500), (40, 40)], dim=dim, dtype=dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    c.cache.v.fill_(0x88)
    s = (1 + torch.rand(c.cache.v_scale.shape[:-1], generator=g, device="cuda")).to(BF)
    c.cache.v_scale[..., 0], c.cache.v_scale[..., 1] = s, -8 * s
    assert not bool(c.attend(window=window)["out"].any())


def check_few_keys(c, window=0):
    """Rows that see at most 512 keys: a weight is the sum of two fp16 numbers, the second the first
    one's rounding error rounded, at most 2^-11 of 2^-11 off.  Others: one number.

    Every 16th key weighs 1 and holds zeros.  The rest weigh w = 0.7107 and hold 7, or w^2 and -8,
    such that sums stay within 8 of nothing; fp16 rounds w up by 3.3e-4 of it and w^2 down by
    4.2e-4, so that roundings add up where the values cancel.  Scores are few powers of w, so each of
    their four operations is 2^-23 off at most, an exponential 2 ulp; sums of n terms n 2^-23."""
    w = 0.7107
    c.q = torch.ones_like(c.q)
    c.cache.k.zero_()
    c.cache.k_scale[..., 0] = 2.0 ** -120
    c.cache.v_scale[..., 0], c.cache.v_scale[..., 1] = 1.0, -8.0
    longest = max(L for _, L in c.lens)
    level, value, total = [], [], 0.0
    for j in range(longest):
        up = total <= 0
        level.append(0 if j % 16 == 0 else 1 if up else 2)
        value.append(0 if j % 16 == 0 else 7 if up else -8)
        total += value[-1] * w ** level[-1]
    level, value = (torch.tensor(x, device="cuda").double() for x in (level, value))
    p, want, mass, low, seen = w ** level, [], [], [], []
    for b, (n, L) in enumerate(c.lens):
        j = torch.arange(L, device="cuda")
        page = torch.tensor(c.owned[b] + [0], device="cuda")[j // c.ps]
        c.cache.k_scale[page, :, j % c.ps, 1] = -level[:L, None].to(BF)
        c.cache.v[page, :, j % c.ps] = (17 * (value[:L] + 8)).to(torch.uint8)[:, None, None]
        hi = L - n + 1 + torch.arange(n, device="cuda")
        lo = (hi - window).clamp(min=0) if window else torch.zeros_like(hi)
        sums = [torch.nn.functional.pad(x.cumsum(0), (1, 0)) for x in (p, p * value, p * value.abs())]
        l, t, m = (x[hi] - x[lo] for x in sums)
        low.append(l)
        want.append(t / l)
        mass.append(m / l)
        seen.append(hi - lo)
    want, mass, seen, low = (torch.cat(x)[:, None] for x in (want, mass, seen, low))
    o = c.attend(window=window, scale=-math.log(w) / c.D)
    tol = HALF[FP] * want.abs() + TINY[FP] + mass * (2.0 ** -22 + 2.0 ** -19 + seen * 2.0 ** -23)
    tol = torch.where(seen <= 512, tol, tol + mass * 2.0 ** -11)
    err = (o["out"].double() - want[..., None]).abs()
    assert bool((err <= tol[..., None]).all()), f"out off by {float((err / tol[..., None]).max()):.2f} of its bound"
    # a mass of l's roundings, and the logarithm's
    assert bool(((o["lse"].double() - low.log()).abs() <= 2.0 ** -18 + seen * 2.0 ** -23).all())


@pytest.mark.parametrize("pages", [0, 900])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("group", [1, 4, 24, 25, 32, 33, 48, 65, 80])
def test_few_keys_by_groups_and_tables(group, dim, pages):
    """Whatever the group, and however many pages the tables have room for."""
    c = CaseU4([(1, 22), (3, 300), (40, 512), (0, 7), (6, 700)], group=group, dim=dim, kv_heads=1, dtype=FP)
    if pages:
        c.table = torch.nn.functional.pad(c.table, (0, pages), value=2 ** 30)
    check_few_keys(c)


@pytest.mark.parametrize("others", [[], [(1, 3)] * 40, [(400, 1700)], [(1, 900), (150, 160)]])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [16, 496, 511, 512, 513])
def test_few_keys_in_windows_and_company(window, dim, others):
    """A row's accuracy does not go by what else is in the batch."""
    check_few_keys(CaseU4([(1, 2000), (4, 1500), (30, 800), *others], group=4, dim=dim, dtype=FP), window)
