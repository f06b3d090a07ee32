"""Attention over 4-bit pools of unusual contents: steps of either sign, as a pool that was filled
elsewhere may hold, and zero rows among keys of very large products."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged_u4 import BF, FP, CaseU4, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


def hold(c, name, b, sz):
    """Sequence b's steps and zeros [L, H, 2] into c's pool; bounds go by the steps' size."""
    scales, store = (c.cache.k_scale, c.k64) if name == "k" else (c.cache.v_scale, c.v64)
    j = torch.arange(sz.shape[0], device="cuda")
    page = torch.tensor(c.owned[b] + [0], device="cuda")[j // c.ps]
    scales[page, :, j % c.ps] = sz
    store[b] = values(c.c[name][b], sz)
    c.sz[name][b] = torch.stack([sz[..., 0].abs(), sz[..., 1]], -1)


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("signs", ["all", "some"])
@pytest.mark.parametrize("n,dim,dtype", [(1, 64, BF), (5, 128, FP), (40, 64, FP), (40, 128, BF), (10, 128, FP),
                                         (3, 160, BF)])
def test_steps_below_zero(n, dim, dtype, signs, which):
    c = CaseU4([(n, 700), (n, n + 130)], dim=dim, dtype=dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    for name in ("k", "v"):
        if which not in (name, "both"):
            continue
        for b in range(2):
            sz = c.sz[name][b].clone()
            down = torch.rand(sz.shape[:-1], generator=g, device="cuda") < (2.0 if signs == "all" else 0.4)
            sz[..., 0] = torch.where(down, -sz[..., 0], sz[..., 0])
            sz[..., 1] = torch.where(down, -sz[..., 1], sz[..., 1])
            hold(c, name, b, sz)
    c.check()


@pytest.mark.parametrize("step", [0.0, 2.0 ** -120])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 40])
@pytest.mark.parametrize("n,dim", [(1, 64), (1, 128), (40, 64), (10, 128), (40, 128)])
def test_zero_rows_among_large_products(n, dim, size, step):
    """q.k around -2^38 or -2^58 and a scale that brings them back to -8; some later keys are zeros,
    as bad pages read and appended zeros are held: they outweigh the rest.  (As many sequences as it
    takes for a CTA to have several tiles of one.)"""
    c = CaseU4([(n, 700)] * 40 + [(n, n + 430)], dim=dim)
    c.q = -c.q.abs() * 2.0 ** 8
    for b in range(41):
        sz = (c.sz["k"][b].double() * size).to(BF)
        sz[..., 1].abs_()
        sz[300::71] = torch.tensor([step, 0.0], device="cuda").to(BF)
        hold(c, "k", b, sz)
    c.check(scale=1.28 / dim / size / 2.0 ** 8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", [2.0 ** -116, 2.0 ** -100, 2.0 ** -64, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("n,dim", [(1, 64), (5, 128), (10, 128), (40, 128)])
def test_keys_of_any_size(n, dim, size, zeros):
    """Keys far from 1 and a scale that brings their products back, with zeros among them or not."""
    c = CaseU4([(n, 700)] * 40 + [(n, n + 430)], dim=dim)
    for b in range(41):
        sz = (c.sz["k"][b].double() * size).to(BF)
        if zeros:
            sz[300::71] = 0.0
        hold(c, "k", b, sz)
    c.check(scale=dim ** -0.5 / size)


@pytest.mark.parametrize("q_size,k_size", [(2.0 ** -100, 2.0 ** -20), (2.0 ** -60, 2.0 ** -57), (2.0 ** 50, 2.0 ** 60)])
@pytest.mark.parametrize("n,dim", [(1, 64), (5, 128), (10, 128), (40, 128)])
def test_products_of_any_size(n, dim, q_size, k_size):
    """Queries and keys far from 1, rows of queries of very different sizes, zeros among the keys."""
    c = CaseU4([(n, 700)] * 40 + [(n, n + 430)], dim=dim)
    c.q.mul_(q_size)
    c.q[:, 1].mul_(2.0 ** -20)
    c.q[::3, 2] = 0
    for b in range(41):
        sz = (c.sz["k"][b].double() * k_size).to(BF)
        sz[300::71] = 0.0
        hold(c, "k", b, sz)
    c.check(scale=dim ** -0.5 / k_size / q_size)
