"""Host-side refusals of 4-bit caches and of spec_kv_append_rope, and what the binding does with
them before a call is queued (no GPU).  Pointers are made-up addresses that are never dereferenced."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from speculative_decoding_verification_21_gb300 import _lib
from tests import _fake_cuda as fake

A, MIS = 0x10000, 0x10004
ARG, DTYPE, ALIGN, UNSUP = -1, -2, -3, -6
U4 = _lib.SV_U4


def cache(**kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, num_pages=10, page_stride=2 * 16 * 64,
             head_stride=16 * 64, token_stride=64, kv_heads=2, page_size=16, head_dim=64, dtype=U4)
    d.update(kw)
    return _lib._CacheStruct(**d)


def batch(**kw):
    d = dict(block_table=A, q_start=A, kv_len=A, total=8, B=2, max_pages=4)
    d.update(kw)
    return _lib._BatchStruct(**d)


def rope(**kw):
    d = dict(cos_sin=A, positions=100, rot_dim=64, interleaved=0)
    d.update(kw)
    return _lib._RopeStruct(**d)


def ref(s):
    return None if s is None else ctypes.addressof(s)


def append(c, b=None, dtype=1):
    b = b or batch()
    return sv.load().spec_kv_append(ref(c), ref(b), A, A, dtype, 128, 64, None, None)


def read(c, dtype=1):
    return sv.load().spec_kv_read(ref(c), A, A, A, 0, 4, 8, A, A, dtype, None, None)


def attend(c, b=None, dtype=1, heads=8):
    b = b or batch()
    return sv.load().spec_chunk_attention(ref(c), ref(b), A, dtype, heads, 512, 64, 0.125, 0, A, None,
                                          None, A, 1 << 40, None)


def append_rope(c=None, b=None, r=None, k=A, v=A, dtype=1, ts=128, hs=64, q=A, heads=8, qts=512, qhs=64,
                out_q=A, null=()):
    c, b, r = c or cache(), b or batch(), r or rope()
    at = {"c": ref(c), "b": ref(b), "r": ref(r)}
    at.update({x: None for x in null})
    return sv.load().spec_kv_append_rope(at["c"], at["b"], at["r"], k, v, dtype, ts, hs, q, heads, qts, qhs,
                                         out_q, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k_scale=None), ARG), (dict(v_scale=None), ARG), (dict(k_scale=A + 2), ALIGN),
    (dict(v_scale=A + 1), ALIGN), (dict(head_dim=16), UNSUP), (dict(head_dim=80), UNSUP),
    (dict(head_dim=288), UNSUP), (dict(k=MIS), ALIGN), (dict(token_stride=48), ALIGN),
    (dict(token_stride=65), ALIGN), (dict(head_stride=16), ALIGN), (dict(page_stride=-32), ARG),
    (dict(v=None), ARG), (dict(dtype=6), DTYPE),
])
def test_bad_caches(kw, status):
    c = cache(**kw)
    assert append(c) == status
    assert read(c) == status
    assert attend(c) == status
    assert append_rope(c) == status
    assert sv.load().sv_attention_workspace_bytes(ref(c), 8) == 0


def test_rows_of_either_type_and_empty_calls():
    for dtype in (1, 2):
        assert append(cache(), batch(B=0), dtype) == 0
        assert attend(cache(), batch(B=0), dtype) == 0
        assert read(cache(), dtype) == 0
        assert append_rope(b=batch(B=0), dtype=dtype) == 0
    assert append(cache(), dtype=0) == DTYPE and append(cache(), dtype=U4) == DTYPE
    assert append_rope(dtype=3) == DTYPE


def test_rope_refusals():
    for x in "cbr":
        assert append_rope(null=(x,)) == ARG
    assert append_rope(k=None) == ARG and append_rope(v=None) == ARG
    assert append_rope(q=None) == ARG and append_rope(out_q=None) == ARG
    assert append_rope(heads=-1) == ARG
    assert append_rope(b=batch(total=2 ** 30), heads=2) == UNSUP
    assert append_rope(k=A + 8) == ALIGN and append_rope(q=A + 8) == ALIGN
    assert append_rope(out_q=A + 8) == ALIGN
    assert append_rope(ts=130) == ALIGN and append_rope(qts=516) == ALIGN and append_rope(qhs=-8) == ARG
    assert append_rope(r=rope(cos_sin=None)) == ARG
    assert append_rope(r=rope(cos_sin=MIS)) == ALIGN
    assert append_rope(r=rope(positions=-1)) == ARG
    assert append_rope(r=rope(positions=2 ** 31)) == ARG
    assert append_rope(r=rope(rot_dim=0)) == ARG
    assert append_rope(r=rope(rot_dim=-16)) == ARG
    assert append_rope(r=rope(rot_dim=80)) == ARG        # more than the head has
    assert append_rope(r=rope(rot_dim=24)) == UNSUP
    assert append_rope(r=rope(interleaved=2)) == ARG
    assert append_rope(b=batch(q_start=None)) == ARG
    assert append_rope(c=cache(dtype=2, k_scale=None, v_scale=None)) == DTYPE  # bf16 rows, fp16 cache
    # (keys and values alone need no queries; no sequences need nothing)
    assert append_rope(b=batch(B=0), q=None, out_q=None, heads=0) == 0
    assert append_rope(b=batch(B=0), r=rope(cos_sin=None), k=None, v=None) == 0


@pytest.fixture
def cuda(monkeypatch):
    return fake.Cuda(monkeypatch)


BF, F32 = torch.bfloat16, torch.float32


def fake_cache(device="cuda:0", **kw):
    d = {"k": fake.Tensor((10, 2, 16, 32), torch.uint8, device), "v": fake.Tensor((10, 2, 16, 32), torch.uint8, device),
         "k_scale": fake.Tensor((10, 2, 16, 2), BF, device), "v_scale": fake.Tensor((10, 2, 16, 2), BF, device)}
    d.update(kw)
    return _lib.KVCache(**d)


def rows(shape=(6, 2, 64), dtype=BF, device="cuda:0", **kw):
    return fake.Tensor(shape, dtype, device, **kw)


def call(device="cuda:0", **kw):
    t, s, n = fake.index_arrays(device)
    a = {"cache": fake_cache(device), "new_k": rows(device=device), "new_v": rows(device=device),
         "block_table": t, "q_start": s, "kv_len": n, "cos_sin": rows((100, 64), F32, device),
         "q": rows((6, 8, 64), device=device)}
    a.update(kw)
    return _lib.spec_kv_append_rope(**a)


def test_a_cache_of_codes(cuda):
    c = fake_cache()
    assert c.head_dim == 64 and c._struct.head_dim == 64 and c._struct.dtype == U4
    assert (c._struct.page_stride, c._struct.head_stride, c._struct.token_stride) == (2048, 1024, 64)
    for kw in (dict(k_scale=None), dict(v_scale=None),
               dict(k_scale=fake.Tensor((10, 2, 16), BF)), dict(v_scale=fake.Tensor((10, 2, 16, 2), F32)),
               dict(k_scale=fake.Tensor((10, 2, 16, 2), BF, strides=(128, 64, 4, 2))),
               dict(v_scale=fake.Tensor((10, 2, 16, 2), BF, "cuda:1")),
               dict(v=fake.Tensor((10, 2, 16, 32), torch.uint8, "cuda:1")),
               dict(v=fake.Tensor((10, 2, 16, 64), torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            fake_cache(**kw)
    assert sv.alloc_kv_cache(3, 2, 16, 96, dtype=torch.uint8).head_dim == 96
    with pytest.raises(ValueError):
        sv.alloc_kv_cache(3, 2, 16, 33, dtype=torch.uint8)


def test_outputs_of_a_read_of_codes(cuda):
    t, s, n = fake.index_arrays()
    r = _lib.spec_kv_read(fake_cache(), t, n, s, 6)
    assert r["k"].dtype == BF and tuple(r["k"].shape) == (6, 2, 64)
    assert _lib.spec_kv_read(fake_cache(), t, n, s, 6, dtype=torch.float16)["v"].dtype == torch.float16


def test_rope_arguments(cuda):
    r = call(want_flags=True)
    assert set(r) == {"q", "flags"} and tuple(r["q"].shape) == (6, 8, 64) and r["q"].dtype == BF
    name, args, device = cuda.library.calls[-1]
    assert name == "spec_kv_append_rope" and device == 0
    assert args[5:8] == (1, 128, 64) and args[9:12] == (8, 512, 64)
    r = call(q=None)
    assert r == {} and cuda.library.calls[-1][1][8:13] == (None, 0, 0, 0, None)
    mine = rows((6, 8, 64))
    assert call(q=mine, out={"q": mine})["q"] is mine
    n = len(cuda.library.calls)
    for kw in (dict(new_v=rows(dtype=torch.float16)), dict(new_v=rows((5, 2, 64))), dict(new_k=rows((6, 3, 64))),
               dict(new_k=rows((6, 2, 32)), new_v=rows((6, 2, 32))), dict(q=rows((5, 8, 64))),
               dict(q=rows((6, 8, 64), torch.float16)), dict(q=rows((6, 8, 32))),
               dict(q=rows((6, 8, 64), device="cuda:1")), dict(cos_sin=rows((100, 64), F32, "cuda:1")),
               dict(cos_sin=rows((100, 64), BF)), dict(cos_sin=rows((6400,), F32)),
               dict(cos_sin=rows((100, 64), F32, strides=(128, 1))), dict(q_start=fake.Tensor((2,), torch.int32)),
               dict(kv_len=fake.Tensor((2,), torch.int64)), dict(out={"q": None}),
               dict(out={"q": rows((6, 8, 64), torch.float16)}), dict(out={"q": rows((5, 8, 64))}),
               dict(out={"q": rows((6, 8, 64), strides=(1024, 64, 1))}), dict(out={"q": rows((6, 8, 64), device="cuda:1")}),
               dict(out={"flags": fake.Tensor((1,), torch.uint8)}), dict(new_k=rows((6, 2, 64), strides=(256, 128, 2)),
                                                                         new_v=rows((6, 2, 64), strides=(256, 128, 2))),
               dict(stream=fake.Stream("elsewhere", "cuda:1"))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    assert len(cuda.library.calls) == n


def test_rope_streams_and_devices(cuda):
    side = fake.Stream("side")
    cuda.made.clear()
    call(stream=side, want_flags=True)
    assert cuda.library.calls[-1][1][-1] == side.cuda_stream
    assert cuda.made and all(t.made_under is side and not t.filled for t in cuda.made)
    assert all(t.recorded == [cuda.default[0]] for t in cuda.made)
    call("cuda:1")
    assert cuda.library.calls[-1][2] == 1 and cuda.library.calls[-1][1][-1] == cuda.default[1].cuda_stream
