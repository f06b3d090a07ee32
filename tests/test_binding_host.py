"""What the binding does on the host before a call is queued: memory by stream, workspaces that
grow, refusals (no GPU)."""
import threading
import time
import weakref

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_verification_21_gb300 import _lib
from tests import _fake_cuda as fake


@pytest.fixture
def cuda(monkeypatch):
    return fake.Cuda(monkeypatch)


@pytest.mark.parametrize("name", fake.NAMES)
def test_memory_of_a_call_belongs_to_the_stream_it_is_queued_on(cuda, name):
    """Outputs and workspace are allocated under `stream`, not filled, and noted as used by the
    caller's stream: a fill, or another tensor's last use, is otherwise ordered on a stream that
    the call does not wait for."""
    call = fake.calls()[name]
    side = fake.Stream("side")
    cuda.made.clear()
    call(stream=side, **fake.FLAGS[name])
    handle = cuda.library.calls[-1][1][-1]
    assert getattr(handle, "value", handle) == side.cuda_stream
    assert cuda.made and all(t.made_under is side for t in cuda.made)
    assert not any(t.filled for t in cuda.made)
    assert all(t.recorded == [cuda.default[0]] for t in cuda.made)


@pytest.mark.parametrize("name", fake.NAMES)
def test_memory_of_a_call_on_the_current_stream(cuda, name):
    call = fake.calls()[name]
    side = fake.Stream("side")
    with cuda.stream(side):
        cuda.made.clear()
        call()
        call(stream=side)
    assert all(t.made_under is side and not t.filled and not t.recorded for t in cuda.made)


def test_an_outgrown_workspace_is_kept():
    """A captured graph, or a call that another stream has not passed, may still use it."""
    cache, cpu = _lib._WorkspaceCache(), torch.device("cpu")
    sizes = [1000, 1001, 3000, 50000]
    bufs = [weakref.ref(cache.get(n, cpu, 7)) for n in sizes]
    assert all(b() is not None and b().numel() >= n for b, n in zip(bufs, sizes))
    assert cache.get(10, cpu, 7) is bufs[-1]()  # calls share the largest
    assert cache.get(10, cpu, 8) is not bufs[-1]()


def test_outgrown_workspaces_take_no_more_than_the_one_in_use():
    cache, cpu = _lib._WorkspaceCache(), torch.device("cpu")
    seen = {}
    for n in range(300, 40000, 97):
        b = cache.get(n, cpu, 7)
        seen[b.data_ptr()] = b.numel()
    assert sum(seen.values()) <= 2 * b.numel()


def attention_outputs(**change):
    o = {"out": fake.Tensor((6, 8, 64), fake.BF), "lse": fake.Tensor((6, 8), fake.F32),
         "flags": fake.Tensor((2,), torch.uint8)}
    return {**o, **change}


def probs_outputs(**change):
    o = {"tokens": fake.Tensor((2, 5), fake.I32), "counts": fake.Tensor((2,), fake.I32),
         "flags": fake.Tensor((2,), torch.uint8)}
    return {**o, **change}


def rows_outputs(**change):
    o = {"k": fake.Tensor((6, 2, 64), fake.BF), "v": fake.Tensor((6, 2, 64), fake.BF),
         "flags": fake.Tensor((2,), torch.uint8)}
    return {**o, **change}


def flags_only(**change):
    return {"flags": fake.Tensor((2,), torch.uint8), **change}


NEW = {"spec_chunk_attention": attention_outputs, "spec_verify_probs": probs_outputs,
       "spec_kv_read": rows_outputs, "spec_kv_append": flags_only}


@pytest.mark.parametrize("name", NEW)
def test_outputs_that_are_handed_in_are_looked_at(cuda, name):
    """A short tensor, or one of a narrower type, would be written past its end."""
    call, outputs = fake.calls()[name], NEW[name]
    r = call(out=outputs(), want_flags=True)
    assert set(r) == set(outputs()) and len(cuda.library.calls) == 1
    for key, good in outputs().items():
        shape, dtype = tuple(good.shape), good.dtype
        wrong_type = torch.int8 if dtype != torch.int8 else torch.uint8
        for bad in (fake.Tensor((shape[0] - 1,) + shape[1:], dtype),          # short
                    fake.Tensor(shape[:-1] + (shape[-1] + 1,), dtype),        # another shape
                    fake.Tensor(shape + (1,), dtype),
                    fake.Tensor(shape, torch.float64 if dtype != torch.float64 else dtype),
                    fake.Tensor(shape, wrong_type),                           # narrower
                    fake.Tensor(shape, dtype, strides=[2 * s for s in good.stride()]),
                    fake.Tensor(shape, dtype, "cpu")):
            with pytest.raises((ValueError, TypeError)):
                call(out=outputs(**{key: bad}))
    assert len(cuda.library.calls) == 1


@pytest.mark.parametrize("name", [n for n in fake.NAMES if n not in NEW])
def test_older_calls_refuse_outputs_without_room(cuda, name):
    call = fake.calls()[name]
    full = call(**fake.FLAGS[name])
    n = len(cuda.library.calls)
    call(out=full)
    for key, t in full.items():
        size = t.numel()
        call(out={**full, key: fake.Tensor((size,), t.dtype)})  # (any shape will do)
        for bad in (fake.Tensor((size - 1,), t.dtype), fake.Tensor((size,), t.dtype, "cpu"),
                    fake.Tensor((size,), t.dtype, strides=(2,))):
            with pytest.raises(ValueError):
                call(out={**full, key: bad})
    assert len(cuda.library.calls) == n + 1 + len(full)


def test_workspaces_that_are_handed_in_are_looked_at(cuda):
    for name, call in fake.calls().items():
        if name in ("spec_kv_append", "spec_kv_read", "spec_verify_probs"):
            continue  # (need none)
        call(workspace=fake.Tensor((5000,), torch.uint8))
        assert cuda.library.calls[-1][1][-2] == 5000
        for bad in (fake.Tensor((5000,), torch.uint8, "cpu"),
                    fake.Tensor((5000,), torch.uint8, strides=(2,))):
            with pytest.raises(ValueError):
                call(workspace=bad)


@pytest.mark.parametrize("name", fake.NAMES)
def test_tensors_of_two_devices_are_refused(cuda, name):
    for device, other in (("cuda:0", "cuda:1"), ("cuda:1", "cuda:0")):
        with pytest.raises(ValueError):
            fake.calls(device, other)[name]()
    with pytest.raises(ValueError):
        fake.calls()[name](stream=fake.Stream("elsewhere", "cuda:1"))
    t, q_start, kv_len = fake.index_arrays()
    k, v = (fake.Tensor((6, 2, 64), fake.BF, d) for d in ("cuda:0", "cuda:1"))
    for new in ((k, v), (v, k), (v, v)):
        with pytest.raises(ValueError):
            _lib.spec_kv_append(fake.cache(), *new, t, q_start, kv_len)
    assert not cuda.library.calls


def test_a_cache_has_one_device(cuda):
    k, far = (fake.Tensor((10, 2, 16, 64), fake.BF, d) for d in ("cuda:0", "cuda:1"))
    with pytest.raises(ValueError):
        _lib.KVCache(k, far)
    codes = [fake.Tensor((10, 2, 16, 64), torch.float8_e4m3fn) for _ in range(2)]
    near, far = (fake.Tensor((10, 2, 16), torch.uint8, d) for d in ("cuda:0", "cuda:1"))
    for scales in ((near, far), (far, near), (far, far)):
        with pytest.raises(ValueError):
            _lib.KVCache(*codes, *scales)
    _lib.KVCache(*codes, near, near)


@pytest.mark.parametrize("name", fake.NAMES)
def test_a_call_is_queued_on_its_tensors_device(cuda, name):
    """The library launches on the current device."""
    call = fake.calls("cuda:1")[name]
    call()
    entry, args, device = cuda.library.calls[-1]
    assert device == 1 and cuda.device_index == 0
    handle = getattr(args[-1], "value", args[-1])
    assert handle == cuda.default[1].cuda_stream
    assert all(t.made_under is cuda.default[1] for t in cuda.made)


def test_a_window_past_32_bits_hides_nothing(cuda):
    """(It would be cut to its low 32 bits on the way to the library.)"""
    attend = fake.calls()["spec_chunk_attention"]
    for window, passed in ((0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                           (2 ** 32 + 5, 2 ** 31 - 1), (10 ** 12, 2 ** 31 - 1)):
        attend(window=window)
        assert cuda.library.calls[-1][1][8] == passed
    for window in (-1, -2 ** 31, -2 ** 32 - 5):  # the library refuses what is negative
        attend(window=window)
        assert cuda.library.calls[-1][1][8] == -1


def test_calls_of_two_threads_do_not_interleave_on_the_device(cuda, monkeypatch):
    """Calls of a stream share its workspace, and one call queues several kernels: another's in
    between would use the workspace too.  (ctypes lets other threads run during a call.)"""
    inside, most = [], []

    class Slow(fake.Library):
        def __getattr__(self, name):
            def entry(*args):
                if name.endswith("workspace_bytes"):
                    return 5000
                inside.append(name)
                most.append(len(inside))
                time.sleep(0.002)
                inside.pop()
                return 0
            return entry

    monkeypatch.setattr(_lib, "_lib", Slow(cuda))
    calls = [fake.calls()[n] for n in ("spec_chunk_attention", "spec_verify", "spec_kv_append")]
    threads = [threading.Thread(target=lambda c=c: [c() for _ in range(10)]) for c in calls * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 60 and max(most) == 1
