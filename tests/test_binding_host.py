"""What the binding does on the host before a call is queued: memory by stream (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

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
