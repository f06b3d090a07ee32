"""Attention over 4-bit codes on both sides of the rule that tells the kernel of few rows from that
of many: the table's or the window's keys, and how much of an item's rows a group fills."""
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


def case(n, keys, **kw):
    """Chunks of n tokens, tables of just so many keys."""
    c = CaseU4([(n, 900), (n, n + 70), (1, 5)], page=32, **kw)
    more = keys // c.ps - c.table.shape[1]
    c.table = torch.nn.functional.pad(c.table, (0, more), value=2 ** 30).contiguous()
    assert c.table.shape[1] * c.ps == keys
    return c


@pytest.mark.parametrize("dim,keys", [(32, 3200), (64, 4096), (96, 2048)])
@pytest.mark.parametrize("over", [0, 32])
@pytest.mark.parametrize("group,n", [(1, 60), (5, 17), (8, 100)])
def test_tables_around_the_bound(dim, keys, over, group, n):
    for dtype in (BF, FP):
        case(n, keys + over, group=group, dim=dim, dtype=dtype).check()


@pytest.mark.parametrize("dim,window", [(32, 3150), (32, 3201), (64, 4000), (64, 4097), (96, 2000), (96, 2049)])
def test_windows_around_the_bound(dim, window):
    CaseU4([(40, 5000), (30, 300)], dim=dim, group=4, page=32).check(window=window)


@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("group", [9, 10, 11, 12, 13, 16, 17, 20, 23, 24, 26, 27, 32, 33, 40, 41, 48, 49])
def test_groups_that_fill_an_item_or_do_not(group, dim):
    case(9, 1024, group=group, dim=dim, kv_heads=1).check()
