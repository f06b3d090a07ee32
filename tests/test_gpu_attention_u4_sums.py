"""What sums over 4-bit values lose: codes are centred before they are multiplied, so neither the
sums' last bits nor the weights' roundings grow with values that cancel."""
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
