"""Failure detection of the attention's tile kernel without a GPU fault.

A bounded wait is made to run out on purpose: one CTA never hands its first scores to the softmax
(sv_test_attention_stall), whose wait gives up after a short limit.  The CTA ends its other
roles, lets its copies land, frees its tensor memory and returns; the call returns normally with
every sequence flagged SV_FLAG_TIMEOUT, and the next call on the same context gives the results
of a call that never stalled.
"""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import Case, E4M3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("lens", [[(1, 300)], [(5, 4000), (200, 900), (1, 20)]])
def test_stalled_scores_time_out_and_the_context_survives(lens, cache):
    c = Case(lens, dim=128, cache=cache)
    want = c.attend(want_flags=True)
    assert not bool(want["flags"].any())
    sv.test_attention_stall(3, 1 << 22)  # (an item's start counts three tiles: CTA 3 has the first)
    try:
        stalled = c.attend(want_flags=True)
        torch.cuda.synchronize()
    finally:
        sv.test_attention_stall(-1, 0)
    assert bool((stalled["flags"] & sv.FLAG_TIMEOUT).all())
    for _ in range(3):
        again = c.attend(want_flags=True)
        assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])
        assert not bool(again["flags"].any())


def test_the_workspace_names_the_cta_and_the_wait_that_gave_up():
    c = Case([(5, 4000), (200, 900)], dim=128)
    ws = torch.zeros(sv.attention_workspace_bytes(c.cache, 8), dtype=torch.uint8, device="cuda")
    err = ws[160 * 16:160 * 20].view(torch.int32)  # (behind 160 records of 16 bytes)
    c.attend(workspace=ws)
    assert not bool(err.any())
    sv.test_attention_stall(3, 1 << 22)
    try:
        c.attend(workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.test_attention_stall(-1, 0)
    e = err.tolist()
    assert e[3] & 1 and 1 <= e[3] >> 8 <= 11
    assert not any(e[:3] + e[4:])
