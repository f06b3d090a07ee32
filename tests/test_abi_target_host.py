"""Host-side refusals of the target's cache, attention and verification entry points (no GPU).

Pointers are made-up addresses that are never dereferenced: every call here returns before
anything is queued."""
import ctypes

import pytest

import speculative_decoding_verification_21_gb300 as sv
from speculative_decoding_verification_21_gb300 import _lib

A = 0x10000       # aligned
MIS = 0x10004     # 4-byte aligned only
ARG, DTYPE, ALIGN, WS, UNSUP = -1, -2, -3, -4, -6


def cache(**kw):
    d = dict(k=A, v=A, k_scale=None, v_scale=None, num_pages=10, page_stride=2 * 16 * 64,
             head_stride=16 * 64, token_stride=64, kv_heads=2, page_size=16, head_dim=64, dtype=1)
    d.update(kw)
    return _lib._CacheStruct(**d)


def batch(**kw):
    d = dict(block_table=A, q_start=A, kv_len=A, total=8, B=2, max_pages=4)
    d.update(kw)
    return _lib._BatchStruct(**d)


def ref(s):
    return None if s is None else ctypes.addressof(s)


def append(c, b, k=A, v=A, dtype=1, ts=128, hs=64, flags=None):
    return sv.load().spec_kv_append(ref(c), ref(b), k, v, dtype, ts, hs, flags, None)


def read(c, table=A, first=A, start=A, B=2, mp=4, total=8, k=A, v=A, dtype=1):
    return sv.load().spec_kv_read(ref(c), table, first, start, B, mp, total, k, v, dtype, None, None)


def attend(c, b, q=A, dtype=1, heads=8, ts=512, hs=64, scale=0.125, window=0, out=A, lse=None,
           ws=A, ws_bytes=1 << 40):
    return sv.load().spec_chunk_attention(ref(c), ref(b), q, dtype, heads, ts, hs, scale, window,
                                          out, lse, None, ws, ws_bytes, None)


def probs(p=A, q=A, x=A, u=A, B=2, g=2, V=64, dtype=0, tok=A, cnt=A):
    return sv.load().spec_verify_probs(p, q, x, u, B, g, V, dtype, tok, cnt, None, None)


CACHES = [
    (None, ARG), (cache(dtype=0), DTYPE), (cache(dtype=4), DTYPE), (cache(kv_heads=0), ARG),
    (cache(page_size=0), ARG), (cache(head_dim=0), ARG), (cache(head_dim=72), UNSUP),
    (cache(head_dim=272), UNSUP), (cache(num_pages=-1), ARG), (cache(num_pages=2 ** 31), ARG),
    (cache(k=None), ARG), (cache(v=None), ARG), (cache(k=MIS), ALIGN), (cache(v=MIS), ALIGN),
    (cache(token_stride=68), ALIGN), (cache(head_stride=-8), ARG), (cache(page_stride=2049), ALIGN),
    (cache(dtype=3), ARG),                                              # e4m3 without scales
    (cache(dtype=3, k_scale=A, v_scale=A, token_stride=72), ALIGN),     # 72 bytes
]
BATCHES = [
    (None, ARG), (batch(B=-1), ARG), (batch(total=-1), ARG), (batch(total=2 ** 31), ARG),
    (batch(max_pages=-1), ARG), (batch(max_pages=2 ** 28), ARG), (batch(q_start=None), ARG),
    (batch(kv_len=None), ARG), (batch(block_table=None), ARG), (batch(q_start=A + 2), ALIGN),
]


@pytest.mark.parametrize("i", range(len(CACHES)))
def test_bad_caches(i):
    c, st = CACHES[i]
    assert append(c, batch()) == st
    assert read(c) == st
    assert attend(c, batch()) == st
    assert sv.load().sv_attention_workspace_bytes(ref(c), 8) == 0


@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_bad_batches(i):
    b, st = BATCHES[i]
    assert append(cache(), b) == st
    assert attend(cache(), b) == st


def test_empty_calls_do_nothing():
    for r in (append(cache(), batch(B=0)), attend(cache(), batch(B=0)), read(cache(), B=0),
              probs(B=0), append(cache(), batch(B=0, block_table=None, q_start=None, kv_len=None))):
        assert r == 0


def test_append_refusals():
    assert append(cache(), batch(), k=None) == ARG
    assert append(cache(), batch(), v=None) == ARG
    assert append(cache(), batch(), k=A + 8) == ALIGN
    assert append(cache(), batch(), ts=130) == ALIGN
    assert append(cache(), batch(), hs=-64) == ARG
    assert append(cache(), batch(), dtype=0) == DTYPE
    assert append(cache(), batch(), dtype=2) == DTYPE       # fp16 rows, bf16 cache
    assert append(cache(), batch(), dtype=3) == DTYPE


def test_read_refusals():
    assert read(cache(), table=None) == ARG
    assert read(cache(), first=None) == ARG
    assert read(cache(), start=None) == ARG
    assert read(cache(), k=None) == ARG
    assert read(cache(), v=A + 8) == ALIGN
    assert read(cache(), dtype=2) == DTYPE
    assert read(cache(), total=-1) == ARG


def test_attention_refusals():
    assert attend(cache(), batch(), q=None) == ARG
    assert attend(cache(), batch(), out=None) == ARG
    assert attend(cache(), batch(), q=A + 8) == ALIGN
    assert attend(cache(), batch(), out=A + 8) == ALIGN
    assert attend(cache(), batch(), lse=A + 2) == ALIGN
    assert attend(cache(), batch(), heads=7) == ARG
    assert attend(cache(), batch(), heads=0) == ARG
    assert attend(cache(), batch(), heads=2 * 129) == UNSUP
    assert attend(cache(), batch(total=2 ** 30)) == UNSUP
    assert attend(cache(), batch(), window=-1) == ARG
    assert attend(cache(), batch(), scale=float("nan")) == ARG
    assert attend(cache(), batch(), scale=float("inf")) == ARG
    assert attend(cache(), batch(), dtype=2) == DTYPE


def test_probs_refusals():
    for name in ("p", "q", "x", "u", "tok", "cnt"):
        assert probs(**{name: None}) == ARG
    assert probs(p=A + 8) == ALIGN
    assert probs(q=A + 4) == ALIGN
    assert probs(x=A + 2) == ALIGN
    assert probs(dtype=2) == DTYPE
    assert probs(g=0) == ARG and probs(g=33) == ARG and probs(V=0) == ARG and probs(B=-1) == ARG


def test_flags_are_distinct_bits():
    f = [sv.FLAG_ZERO_MASS, sv.FLAG_NONFINITE, sv.FLAG_RESIDUAL_FALLBACK, sv.FLAG_TIMEOUT,
         sv.FLAG_BAD_TOKEN, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_LENGTH]
    assert sorted(f) == [1 << i for i in range(7)]


def test_a_scale_that_leaves_the_range_in_log2_units_is_refused():
    """(Scores are kept in log2 units: scale log2 e has to be a float.)"""
    for scale in (3e38, -3e38, 2.36e38):
        assert attend(cache(), batch(), scale=scale) == ARG
    assert attend(cache(), batch(B=0), scale=2.35e38) == 0


def test_rows_whose_last_tile_passes_31_bits_are_refused():
    for total in (2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 1023):
        assert attend(cache(kv_heads=1), batch(total=total), heads=1) == UNSUP
    assert attend(cache(), batch(total=2 ** 30 - 1), heads=2) == UNSUP
    assert attend(cache(kv_heads=1), batch(total=2 ** 31 - 1024, B=0), heads=1) == 0
