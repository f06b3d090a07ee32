"""What the binding does on the host before a call is queued: memory by stream, workspaces that
grow (no GPU)."""
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
