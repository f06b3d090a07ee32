"""Stand-ins for CUDA tensors, streams and the library: what the binding does on the host before a
call is queued, seen without a GPU.  Nothing here computes; addresses are made up."""
import contextlib
import itertools

import torch

from speculative_decoding_verification_21_gb300 import _lib

_addresses = itertools.count(0x100000, 0x100000)


class Stream:
    def __init__(self, name, device="cuda:0"):
        self.name, self.device = name, torch.device(device)
        self.cuda_stream = next(_addresses)


class Tensor:
    def __init__(self, shape, dtype, device="cuda:0", strides=None, made_under=None):
        self.shape = torch.Size(shape)
        self.dtype, self.device = dtype, torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", 0)
        packed = [1] * len(self.shape)
        for i in range(len(self.shape) - 2, -1, -1):
            packed[i] = packed[i + 1] * self.shape[i + 1]
        self._packed = tuple(packed)
        self._strides = self._packed if strides is None else tuple(strides)
        self._at = next(_addresses)
        self.made_under, self.recorded = made_under, []

    is_cuda = property(lambda self: self.device.type == "cuda")

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def is_contiguous(self):
        return self._strides == self._packed

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self._at

    def record_stream(self, stream):
        self.recorded.append(stream)


class Library:
    """Every entry point returns 0 and notes its arguments and the device that was current."""

    def __init__(self, cuda, workspace=5000):
        self.cuda, self.workspace, self.calls = cuda, workspace, []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("workspace_bytes"):
                return self.workspace
            self.calls.append((name, args, self.cuda.device_index))
            return 0
        return entry


class Cuda:
    """The parts of torch that the binding uses, with made-up devices and streams; `made` lists what
    was allocated, in order."""

    def __init__(self, monkeypatch, workspace=5000):
        self.device_index, self.made = 0, []
        self.default = [Stream(f"default of {i}", f"cuda:{i}") for i in range(2)]
        self.current = list(self.default)
        self.library = Library(self, workspace)
        monkeypatch.setattr(_lib, "_lib", self.library)
        monkeypatch.setattr(_lib, "_ws_cache", _lib._WorkspaceCache())
        monkeypatch.setattr(torch, "empty", self.empty)
        monkeypatch.setattr(torch, "zeros", self.filled)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device_index)
        monkeypatch.setattr(torch.cuda, "current_stream", self.current_stream)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "device", self.device)

    def _index(self, device):
        index = None if device is None else torch.device(device).index
        return self.device_index if index is None else index

    def empty(self, *shape, dtype=torch.float32, device="cuda", fill=False):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        index = self._index(device)
        t = Tensor(shape, dtype, torch.device("cuda", index), made_under=self.current[index])
        t.filled = fill
        self.made.append(t)
        return t

    def filled(self, *shape, **kw):
        return self.empty(*shape, fill=True, **kw)

    def current_stream(self, device=None):
        return self.current[self._index(device)]

    @contextlib.contextmanager
    def stream(self, stream):
        index = stream.device.index
        was, was_device = self.current[index], self.device_index
        self.current[index], self.device_index = stream, index
        try:
            yield
        finally:
            self.current[index], self.device_index = was, was_device

    @contextlib.contextmanager
    def device(self, device):
        was, self.device_index = self.device_index, self._index(device)
        try:
            yield
        finally:
            self.device_index = was


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def index_arrays(device="cuda:0", B=2, pages=4):
    """block_table, q_start, kv_len of a batch."""
    return Tensor((B, pages), I32, device), Tensor((B + 1,), I32, device), Tensor((B,), I32, device)


def cache(device="cuda:0"):
    k, v = (Tensor((10, 2, 16, 64), BF, device) for _ in range(2))
    return _lib.KVCache(k, v)


def calls(device="cuda:0", other=None):
    """name -> a call of each entry point on small tensors of `device`; keyword arguments pass on.
    `other`: the device of the arguments that index or describe the rest."""
    other = other or device
    t, s, n = index_arrays(other)
    f = lambda shape, dtype=F32, at=device: Tensor(shape, dtype, at)  # noqa: E731
    c = cache(device)
    x = f((2, 4), I32, other)
    lm = (f((10, 64), BF), f((64, 100), BF), f((8, 64), BF), f((64, 100), BF), x)
    return {
        "spec_verify": lambda **k: _lib.spec_verify(f((2, 5, 100)), f((2, 4, 100)), x, **k),
        "spec_verify_greedy": lambda **k: _lib.spec_verify_greedy(f((2, 5, 100)), x, **k),
        "spec_lmhead_verify": lambda **k: _lib.spec_lmhead_verify(*lm, B=2, gamma=4, **k),
        "spec_lmhead_verify_drafted": lambda **k: _lib.spec_lmhead_verify_drafted(
            *lm, f((2, 4)), f((2, 4)), B=2, gamma=4, **k),
        "spec_lmhead_draft": lambda **k: _lib.spec_lmhead_draft(
            f((2, 64), BF), f((64, 100), BF, other), pos=0, **k),
        "spec_kv_append": lambda **k: _lib.spec_kv_append(
            c, f((6, 2, 64), BF), f((6, 2, 64), BF), t, s, n, **k),
        "spec_kv_read": lambda **k: _lib.spec_kv_read(c, t, n, s, 6, **k),
        "spec_chunk_attention": lambda **k: _lib.spec_chunk_attention(
            f((6, 8, 64), BF), c, t, s, n, **k),
        "spec_verify_probs": lambda **k: _lib.spec_verify_probs(
            f((2, 5, 100)), f((2, 4, 100)), x, f((2, 5), at=other), **k),
    }


NAMES = ("spec_verify", "spec_verify_greedy", "spec_lmhead_verify", "spec_lmhead_verify_drafted",
         "spec_lmhead_draft", "spec_kv_append", "spec_kv_read", "spec_chunk_attention",
         "spec_verify_probs")
FLAGS = {n: {} if n in ("spec_verify_greedy", "spec_lmhead_draft") else {"want_flags": True}
         for n in NAMES}
