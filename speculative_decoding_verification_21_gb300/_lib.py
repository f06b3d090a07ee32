"""ctypes binding of libspecverify (argument marshalling only).

Every step of the verify path runs in the CUDA library; this module turns torch
tensors into device pointers, allocates outputs and the workspace with torch
when the caller does not pass them, and raises on a non-OK status.  There is
no CPU fallback: if the library is missing or fails to load, the call raises.

`stream` (every call): the torch stream that the call is queued on, by default the
current one.  What the call allocates is taken for that stream; order the tensors that
are handed in before it, and keep them until it has passed (Tensor.record_stream).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

from . import build as _build

SV_OK = 0
SV_F32, SV_BF16, SV_F16, SV_E4M3 = 0, 1, 2, 3
SV_MODE_SAMPLE, SV_MODE_GREEDY, SV_MODE_LMHEAD, SV_MODE_DRAFT = 0, 1, 2, 3
FLAG_ZERO_MASS, FLAG_NONFINITE, FLAG_RESIDUAL_FALLBACK, FLAG_TIMEOUT, FLAG_BAD_TOKEN = 1, 2, 4, 8, 16
FLAG_BAD_PAGE, FLAG_BAD_LENGTH = 32, 64

EXPORTS = ("sv_workspace_bytes", "sv_workspace_init", "spec_verify", "spec_verify_opts",
           "spec_verify_greedy", "spec_lmhead_verify", "spec_lmhead_draft",
           "spec_lmhead_verify_drafted", "spec_kv_append", "spec_kv_read", "spec_chunk_attention",
           "spec_verify_probs", "sv_attention_workspace_bytes",
           "sv_set_timing_events", "sv_test_lmhead_stall", "sv_test_attention_stall", "sv_status_string", "sv_version")


class Options(ctypes.Structure):
    """sv_options of include/specverify.h."""
    _fields_ = [("lenience", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("top_p", ctypes.c_float), ("sampler", ctypes.c_int32)]


class _CacheStruct(ctypes.Structure):
    """sv_kv_cache of include/specverify.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _BatchStruct(ctypes.Structure):
    """sv_kv_batch of include/specverify.h."""
    _fields_ = [("block_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("total", ctypes.c_int64), ("B", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


SV_SAMPLER_GUMBEL, SV_SAMPLER_INVERSE = 0, 1
SAMPLERS = {"gumbel": SV_SAMPLER_GUMBEL, "inverse": SV_SAMPLER_INVERSE}


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {status_string(status)} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load the in-tree libspecverify.so (building it with nvcc if absent)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"libspecverify is not built ({path}); run __graft_entry__.build()")
            _build.build()
        L = ctypes.CDLL(path)
        P, I, I64, U64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                  ctypes.c_float, ctypes.c_size_t)
        L.sv_workspace_bytes.argtypes = [I, I, I64, I]
        L.sv_workspace_bytes.restype = SZ
        L.sv_workspace_init.argtypes = [P, SZ, P]
        L.sv_workspace_init.restype = I
        L.spec_verify.argtypes = [P, P, P, I, I, I64, I, F, P, U64, U64, P, P, P, P, P, P, P, SZ, P]
        L.spec_verify.restype = I
        L.spec_verify_opts.argtypes = [P, P, P, I, I, I64, I, F, P, U64, U64, P, P, P, P, P, P,
                                       P, P, SZ, P]
        L.spec_verify_opts.restype = I
        L.spec_verify_greedy.argtypes = [P, P, I, I, I64, I, P, P, P, SZ, P]
        L.spec_verify_greedy.restype = I
        L.spec_lmhead_verify.argtypes = [P, P, I, P, P, I, P, I, I, I64, F, U64, U64, P, P, P, P,
                                         P, P, P, SZ, P]
        L.spec_lmhead_verify.restype = I
        L.spec_lmhead_draft.argtypes = [P, P, I, I, I64, F, U64, U64, I, P, P, P, P, P, P, SZ, P]
        L.spec_lmhead_verify_drafted.argtypes = [P, P, I, P, P, I, P, P, P, I, I, I64, F, U64,
                                                 U64, P, P, P, P, P, P, P, SZ, P]
        L.spec_lmhead_verify_drafted.restype = I
        L.spec_lmhead_draft.restype = I
        L.spec_kv_append.argtypes = [P, P, P, P, I, I64, I64, P, P]
        L.spec_kv_append.restype = I
        L.spec_kv_read.argtypes = [P, P, P, P, I, I, I64, P, P, I, P, P]
        L.spec_kv_read.restype = I
        L.sv_attention_workspace_bytes.argtypes = [P, I]
        L.sv_attention_workspace_bytes.restype = SZ
        L.spec_chunk_attention.argtypes = [P, P, P, I, I, I64, I64, F, I, P, P, P, P, SZ, P]
        L.spec_chunk_attention.restype = I
        L.spec_verify_probs.argtypes = [P, P, P, P, I, I, I64, I, P, P, P, P]
        L.spec_verify_probs.restype = I
        L.sv_set_timing_events.argtypes = [P, I]
        L.sv_set_timing_events.restype = I
        L.sv_test_lmhead_stall.argtypes = [I, ctypes.c_uint32]
        L.sv_test_lmhead_stall.restype = I
        L.sv_test_attention_stall.argtypes = [I, I64]
        L.sv_test_attention_stall.restype = I
        L.sv_status_string.argtypes = [I]
        L.sv_status_string.restype = ctypes.c_char_p
        L.sv_version.argtypes = []
        L.sv_version.restype = I
        _lib = L
        return _lib


def test_lmhead_stall(job: int, wait_limit: int = 0) -> None:
    """Test only: the next fused LM-head calls withhold one accumulator hand-over
    (job < 0: none) and give up every bounded wait after `wait_limit` tries (0: the
    default); see sv_test_lmhead_stall in include/specverify.h."""
    load().sv_test_lmhead_stall(int(job), int(wait_limit))


def test_attention_stall(cta: int, wait_clocks: int = 0) -> None:
    """Test only: the same for spec_chunk_attention; see sv_test_attention_stall in
    include/specverify.h."""
    load().sv_test_attention_stall(int(cta), int(wait_clocks))


def status_string(status: int) -> str:
    return load().sv_status_string(int(status)).decode()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_of(stream, device) -> int:
    """The raw stream that a call is queued on: `stream`, or the device's current one."""
    if stream is None:
        return _torch().cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors of {device}")
    return stream.cuda_stream


def _stream_handle(stream, device):
    return ctypes.c_void_p(_stream_of(stream, device))


_queue_lock = threading.Lock()


def _queue(entry, device, *args):
    """entry(*args) with the tensors' device current: the library launches on that.
    One call at a time: the kernels of two calls on one stream, queued by two threads
    (ctypes lets others run meanwhile), would mix in the workspace that they share."""
    cuda = _torch().cuda
    with _queue_lock:
        if cuda.current_device() == device.index:
            return entry(*args)
        with cuda.device(device):
            return entry(*args)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _check_cuda(*ts, device=None):
    """Contiguous tensors of one CUDA device (`device`, or the first one's)."""
    for t in ts:
        if t is None:
            continue
        at = t.device
        if at != device:
            if not t.is_cuda:
                raise ValueError("all tensors must be CUDA tensors (the library has no CPU path)")
            if device is not None:
                raise ValueError(f"all tensors must be on one device, got {device} and {at}")
            device = at
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _empty(shape, dtype, device, stream=None):
    """Uninitialised memory for a call queued on `stream` (None: the current one).
    torch hands memory out again in the order of the stream it was taken under, so
    it is taken under the call's; the current stream, which the caller will mostly
    read outputs on, is noted as its user too."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if current.cuda_stream == stream.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _output(o, name, shape, dtype, device, stream, want=True, any_shape=False):
    """o[name], made if it is missing and wanted.  One that was handed in has to be
    contiguous, on the inputs' device, and of this shape and type (any_shape: of as
    many bytes): the call writes all of it."""
    if name not in o:
        if want:
            o[name] = _empty(shape, dtype, device, stream)
        return
    t = o[name]
    if t is None:
        return
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"out {name}: contiguous and on the inputs' device ({device})")
    if any_shape:
        if t.numel() * t.element_size() < math.prod(shape) * dtype.itemsize:
            raise ValueError(f"out {name}: too small for {shape} of {dtype}")
    elif tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"out {name}: {shape} of {dtype}, got {tuple(t.shape)} of {t.dtype}")


def _workspace(workspace, nbytes, device, stream_key, stream):
    """The workspace of a call: the caller's, or the stream's."""
    if workspace is None:
        return _ws_cache.get(nbytes, device, stream_key, stream)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: contiguous and on the inputs' device ({device})")
    return workspace


class _WorkspaceCache:
    """Workspaces, one per (device, stream), grown on demand.  Calls queued on
    one stream may share a workspace; the library needs no initial contents.  One
    that became too small is kept: a graph captured with it will use it again.  (So
    a graph that runs beside calls of its capture's stream needs a workspace of its
    own, passed as workspace=.)"""

    def __init__(self):
        self._bufs = {}
        self._outgrown = []
        self._lock = threading.Lock()

    def get(self, nbytes: int, device, stream_key, stream=None):
        key = (str(device), stream_key)
        with self._lock:
            buf = self._bufs.get(key)
            if buf is None or buf.numel() < nbytes:
                if buf is not None:  # twice the size at least: what is kept adds up to less than it
                    self._outgrown.append(buf)
                    nbytes = max(nbytes, 2 * buf.numel())
                buf = _empty((max(nbytes, 256),), _torch().uint8, device, stream)
                self._bufs[key] = buf
            return buf


_ws_cache = _WorkspaceCache()


def workspace_bytes(B: int, gamma: int, V: int, mode: int) -> int:
    return int(load().sv_workspace_bytes(int(B), int(gamma), int(V), int(mode)))


def alloc_workspace(B: int, gamma: int, V: int, mode: int, device="cuda"):
    torch = _torch()
    return torch.zeros(max(workspace_bytes(B, gamma, V, mode), 256), dtype=torch.uint8,
                       device=device)


def spec_verify(target_logits, draft_logits, draft_tokens, *, temperature: float = 1.0,
                row_temperature=None, seed: int = 0, round: int = 0, want_pq: bool = True,
                want_alpha: bool = False, want_flags: bool = True, out=None, workspace=None,
                stream=None, lenience: float = 1.0, top_k: int = 0, top_p: float = 1.0,
                sampler: str = "gumbel"):
    """Sampling verify through the C ABI.  Returns a dict of device tensors:
    tokens [B, g+1] int32, counts [B] int32, p/q [B, g] float32 (if want_pq),
    alpha [B] float32 (if want_alpha), flags [B] uint8 (if want_flags).
    lenience: l in (0, 1] (spec_verify_opts; 1 = the exact round).
    top_k: adjust every row to its k largest logits, ties kept (0 = off).
    top_p: then to its nucleus of probability top_p (1 = off).
    sampler: "gumbel" (the round's contract) or "inverse" (the opt-in inverse
    transform) for the target's own token."""
    torch = _torch()
    L = load()
    B, g1, V = target_logits.shape
    g = g1 - 1
    if tuple(draft_logits.shape) != (B, g, V) or tuple(draft_tokens.shape) != (B, g):
        raise ValueError("shape mismatch: target [B,g+1,V], draft [B,g,V], tokens [B,g]")
    if draft_logits.dtype != target_logits.dtype or draft_tokens.dtype != torch.int32:
        raise TypeError("draft logits must match target dtype; draft tokens must be int32")
    _check_cuda(target_logits, draft_logits, draft_tokens, row_temperature)
    dev = target_logits.device
    o = dict(out or {})
    _output(o, "tokens", (B, g1), torch.int32, dev, stream, any_shape=True)
    _output(o, "counts", (B,), torch.int32, dev, stream, any_shape=True)
    _output(o, "p", (B, g), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "q", (B, g), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "alpha", (B,), torch.float32, dev, stream, want_alpha, any_shape=True)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags, any_shape=True)
    sh = _stream_handle(stream, dev)
    need = workspace_bytes(B, g, V, SV_MODE_SAMPLE)
    ws = _workspace(workspace, need, dev, sh.value, stream)
    opts = Options(float(lenience), int(top_k), float(top_p), SAMPLERS[sampler])
    rc = _queue(L.spec_verify_opts, dev, _ptr(target_logits), _ptr(draft_logits),
                _ptr(draft_tokens), B, g, V, _dtype_code(target_logits), float(temperature),
                _ptr(row_temperature), int(seed) & (2**64 - 1), int(round) & (2**64 - 1),
                _ptr(o["tokens"]), _ptr(o["counts"]), _ptr(o.get("p")), _ptr(o.get("q")),
                _ptr(o.get("alpha")), _ptr(o.get("flags")), ctypes.addressof(opts), _ptr(ws),
                ws.numel(), sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify")
    return o


def spec_verify_greedy(target_logits, draft_tokens, *, out=None, workspace=None, stream=None):
    """Greedy verify through the C ABI.  Returns tokens [B, g+1], counts [B]."""
    torch = _torch()
    L = load()
    B, g1, V = target_logits.shape
    g = g1 - 1
    if tuple(draft_tokens.shape) != (B, g) or draft_tokens.dtype != torch.int32:
        raise ValueError("draft tokens must be int32 [B, gamma]")
    _check_cuda(target_logits, draft_tokens)
    dev = target_logits.device
    o = dict(out or {})
    _output(o, "tokens", (B, g1), torch.int32, dev, stream, any_shape=True)
    _output(o, "counts", (B,), torch.int32, dev, stream, any_shape=True)
    sh = _stream_handle(stream, dev)
    need = workspace_bytes(B, g, V, SV_MODE_GREEDY)
    ws = _workspace(workspace, need, dev, sh.value, stream)
    rc = _queue(L.spec_verify_greedy, dev, _ptr(target_logits), _ptr(draft_tokens), B, g, V,
                _dtype_code(target_logits), _ptr(o["tokens"]), _ptr(o["counts"]), _ptr(ws),
                ws.numel(), sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_greedy")
    return o


def spec_lmhead_verify(h_target, W_target, h_draft, W_draft, draft_tokens, *, B: int,
                       gamma: int, temperature: float = 1.0, seed: int = 0, round: int = 0,
                       want_pq: bool = True, want_flags: bool = True, debug_logits=None,
                       out=None, workspace=None, stream=None):
    """Fused LM heads + sampling verify through the C ABI (bf16 inputs)."""
    torch = _torch()
    L = load()
    Mt, Ht = h_target.shape
    Md, Hd = h_draft.shape
    V = W_target.shape[1]
    if Mt != B * (gamma + 1) or Md != B * gamma or tuple(W_target.shape) != (Ht, V) or \
            tuple(W_draft.shape) != (Hd, V) or tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("shape mismatch in spec_lmhead_verify")
    _check_cuda(h_target, W_target, h_draft, W_draft, draft_tokens, debug_logits)
    dev = h_target.device
    o = dict(out or {})
    _output(o, "tokens", (B, gamma + 1), torch.int32, dev, stream, any_shape=True)
    _output(o, "counts", (B,), torch.int32, dev, stream, any_shape=True)
    _output(o, "p", (B, gamma), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "q", (B, gamma), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags, any_shape=True)
    sh = _stream_handle(stream, dev)
    need = workspace_bytes(B, gamma, V, SV_MODE_LMHEAD)
    ws = _workspace(workspace, need, dev, sh.value, stream)
    rc = _queue(L.spec_lmhead_verify, dev, _ptr(h_target), _ptr(W_target), Ht, _ptr(h_draft),
                _ptr(W_draft), Hd, _ptr(draft_tokens), B, gamma, V, float(temperature),
                int(seed) & (2**64 - 1), int(round) & (2**64 - 1), _ptr(o["tokens"]),
                _ptr(o["counts"]), _ptr(o.get("p")), _ptr(o.get("q")), _ptr(o.get("flags")),
                _ptr(debug_logits), _ptr(ws), ws.numel(), sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_lmhead_verify")
    return o


def spec_lmhead_verify_drafted(h_target, W_target, h_draft, W_draft, draft_tokens, draft_lse,
                               draft_logit, *, B: int, gamma: int, temperature: float = 1.0,
                               seed: int = 0, round: int = 0, want_pq: bool = True,
                               want_flags: bool = True, debug_logits=None, out=None,
                               workspace=None, stream=None):
    """spec_lmhead_verify with the draft rows' statistics from the draft step
    (draft_lse, draft_logit [B, gamma] float32, spec_lmhead_draft's lse and logit)."""
    torch = _torch()
    L = load()
    Mt, Ht = h_target.shape
    Md, Hd = h_draft.shape
    V = W_target.shape[1]
    if Mt != B * (gamma + 1) or Md != B * gamma or tuple(W_target.shape) != (Ht, V) or \
            tuple(W_draft.shape) != (Hd, V) or tuple(draft_tokens.shape) != (B, gamma) or \
            tuple(draft_lse.shape) != (B, gamma) or tuple(draft_logit.shape) != (B, gamma):
        raise ValueError("shape mismatch in spec_lmhead_verify_drafted")
    _check_cuda(h_target, W_target, h_draft, W_draft, draft_tokens, draft_lse, draft_logit,
                debug_logits)
    dev = h_target.device
    o = dict(out or {})
    _output(o, "tokens", (B, gamma + 1), torch.int32, dev, stream, any_shape=True)
    _output(o, "counts", (B,), torch.int32, dev, stream, any_shape=True)
    _output(o, "p", (B, gamma), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "q", (B, gamma), torch.float32, dev, stream, want_pq, any_shape=True)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags, any_shape=True)
    sh = _stream_handle(stream, dev)
    need = workspace_bytes(B, gamma, V, SV_MODE_LMHEAD)
    ws = _workspace(workspace, need, dev, sh.value, stream)
    rc = _queue(L.spec_lmhead_verify_drafted, dev, _ptr(h_target), _ptr(W_target), Ht,
                _ptr(h_draft), _ptr(W_draft), Hd, _ptr(draft_tokens), _ptr(draft_lse),
                _ptr(draft_logit), B, gamma, V, float(temperature), int(seed) & (2**64 - 1),
                int(round) & (2**64 - 1), _ptr(o["tokens"]), _ptr(o["counts"]), _ptr(o.get("p")),
                _ptr(o.get("q")), _ptr(o.get("flags")), _ptr(debug_logits), _ptr(ws), ws.numel(),
                sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_lmhead_verify_drafted")
    return o


def spec_lmhead_draft(h_draft, W_draft, *, pos: int, temperature: float = 1.0, seed: int = 0,
                      round: int = 0, debug_logits=None, out=None, workspace=None,
                      stream=None):
    """Draft LM head + draw of one draft position through the C ABI (bf16 inputs).
    Returns tokens [B] int32, q [B] float32 (q(x)), lse [B] float32, logit [B] float32."""
    torch = _torch()
    L = load()
    B, Hd = h_draft.shape
    V = W_draft.shape[1]
    if tuple(W_draft.shape) != (Hd, V):
        raise ValueError("shape mismatch in spec_lmhead_draft")
    _check_cuda(h_draft, W_draft, debug_logits)
    dev = h_draft.device
    o = dict(out or {})
    _output(o, "tokens", (B,), torch.int32, dev, stream, any_shape=True)
    _output(o, "q", (B,), torch.float32, dev, stream, any_shape=True)
    _output(o, "lse", (B,), torch.float32, dev, stream, any_shape=True)
    _output(o, "logit", (B,), torch.float32, dev, stream, any_shape=True)
    sh = _stream_handle(stream, dev)
    need = workspace_bytes(B, 1, V, SV_MODE_DRAFT)
    ws = _workspace(workspace, need, dev, sh.value, stream)
    rc = _queue(L.spec_lmhead_draft, dev, _ptr(h_draft), _ptr(W_draft), Hd, B, V,
                float(temperature), int(seed) & (2**64 - 1), int(round) & (2**64 - 1), int(pos),
                _ptr(o["tokens"]), _ptr(o["q"]), _ptr(o["lse"]), _ptr(o["logit"]),
                _ptr(debug_logits), _ptr(ws), ws.numel(), sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_lmhead_draft")
    return o


class KVCache:
    """A paged cache: two pools of one shape and one set of strides,
    k, v [num_pages, kv_heads, page_size, head_dim] in bfloat16, float16 or
    float8_e4m3fn, the last dimension contiguous (a token-major pool is passed as
    its transpose), and for float8_e4m3fn k_scale, v_scale [num_pages, kv_heads,
    page_size] uint8, a byte s standing for 2^(s - 127).  Sequences find their
    pages through a block_table [B, max_pages] int32.  The tensors are the
    caller's; this object only names them."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        torch = _torch()
        codes = {torch.bfloat16: SV_BF16, torch.float16: SV_F16, torch.float8_e4m3fn: SV_E4M3}
        if k.dtype not in codes:
            raise TypeError(f"a cache is bfloat16, float16 or float8_e4m3fn, got {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
            raise ValueError("k and v: [num_pages, kv_heads, page_size, head_dim], alike in "
                             "shape, type and strides")
        if k.stride(3) != 1:
            raise ValueError("the head dimension must be contiguous")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn caches, and only there")
        if e4m3:
            for s in (k_scale, v_scale):
                if s.dtype != torch.uint8 or tuple(s.shape) != tuple(k.shape[:3]):
                    raise ValueError("scales: uint8 [num_pages, kv_heads, page_size]")
        if not (k.is_cuda and v.device == k.device):
            raise ValueError("k and v must be CUDA tensors of one device (the library has no CPU path)")
        _check_cuda(k_scale, v_scale, device=k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        self._struct = _CacheStruct(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
            v_scale.data_ptr() if e4m3 else None, k.shape[0], k.stride(0), k.stride(1),
            k.stride(2), k.shape[1], k.shape[2], k.shape[3], codes[k.dtype])
        self._ref = ctypes.addressof(self._struct)
        self._attention_ws = {}  # workspace bytes by query heads


def alloc_kv_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, *, dtype,
                   device="cuda") -> KVCache:
    """A head-major cache of zeros."""
    torch = _torch()
    shape = (num_pages, kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return KVCache(k, v)
    ks, vs = (torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def _row_code(t) -> int:
    code = _row_codes.get(t.dtype)
    if code is None:
        torch = _torch()
        _row_codes[torch.bfloat16], _row_codes[torch.float16] = SV_BF16, SV_F16
        code = _row_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"rows must be bfloat16 or float16, got {t.dtype}")
    return code


_row_codes = {}  # torch dtype -> dtype code


def _address(t):
    """A tensor's address as the plain int that a pointer argument takes."""
    return None if t is None else t.data_ptr()


def _check_rows(t, heads, cache, what):
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads and t.shape[1] != heads):
        raise ValueError(f"{what}: [total, heads, head_dim]")
    if t.device != cache.device:
        raise ValueError(f"{what} is on {t.device}, the cache on {cache.device} "
                         "(the library has no CPU path)")
    if t.stride(2) != 1:
        raise ValueError(f"{what}: the head dimension must be contiguous")


def _check_index(block_table, start, length, device):
    torch = _torch()
    _check_cuda(block_table, start, length, device=device)
    i32 = torch.int32
    if block_table.dtype != i32 or start.dtype != i32 or length.dtype != i32:
        raise TypeError("block_table, q_start and lengths must be int32")
    B = length.shape[0]
    if block_table.dim() != 2 or block_table.shape[0] != B or tuple(start.shape) != (B + 1,):
        raise ValueError("shape mismatch: block_table [B, max_pages], q_start [B+1], lengths [B]")
    return B


def spec_kv_append(cache: KVCache, new_k, new_v, block_table, q_start, kv_len, *,
                   want_flags: bool = False, out=None, stream=None):
    """Write the chunk's keys and values new_k, new_v [total, kv_heads, head_dim]
    (bfloat16 or float16; any token and head strides, alike in both) into the
    cache's pages: sequence b's rows q_start[b] .. q_start[b+1]-1 become its last
    tokens before kv_len[b].  Returns a dict with flags [B] uint8 (if want_flags)."""
    torch = _torch()
    L = _lib or load()
    _check_rows(new_k, cache.kv_heads, cache, "new_k")
    if new_v.shape != new_k.shape or new_v.dtype != new_k.dtype or \
            new_v.stride() != new_k.stride() or new_v.device != cache.device:
        raise ValueError("new_v must match new_k in shape, type, strides and device")
    B = _check_index(block_table, q_start, kv_len, cache.device)
    dev = new_k.device
    o = dict(out or {})
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags)
    batch = _BatchStruct(block_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                         new_k.shape[0], B, block_table.shape[1])
    rc = _queue(L.spec_kv_append, dev, cache._ref, ctypes.addressof(batch), _address(new_k),
                _address(new_v), _row_code(new_k), new_k.stride(0), new_k.stride(1),
                _address(o.get("flags")), _stream_of(stream, dev))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_kv_append")
    return o


def spec_kv_read(cache: KVCache, block_table, first, out_start, total: int, *, dtype=None,
                 want_flags: bool = False, out=None, stream=None):
    """Tokens first[b] .. of every sequence out of the pages, out_start[b+1] -
    out_start[b] of them, packed.  dtype: the cache's own (the default), or either
    16-bit type (default bfloat16) for a float8_e4m3fn cache.  Returns a dict:
    k, v [total, kv_heads, head_dim], flags [B] uint8 (if want_flags)."""
    torch = _torch()
    L = _lib or load()
    B = _check_index(block_table, out_start, first, cache.device)
    if dtype is None:
        dtype = torch.bfloat16 if cache.dtype == torch.float8_e4m3fn else cache.dtype
    dev = cache.device
    o = dict(out or {})
    for name in ("k", "v"):
        _output(o, name, (total, cache.kv_heads, cache.head_dim), dtype, dev, stream)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags)
    rc = _queue(L.spec_kv_read, dev, cache._ref, _address(block_table), _address(first),
                _address(out_start), B, block_table.shape[1], int(total), _address(o["k"]),
                _address(o["v"]), _row_code(o["k"]), _address(o.get("flags")),
                _stream_of(stream, dev))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_kv_read")
    return o


def attention_workspace_bytes(cache: KVCache, heads: int) -> int:
    n = cache._attention_ws.get(heads)
    if n is None:
        n = int(load().sv_attention_workspace_bytes(cache._ref, int(heads)))
        cache._attention_ws[heads] = n
    return n


def spec_chunk_attention(q, cache: KVCache, block_table, q_start, kv_len, *, scale=None,
                         window: int = 0, want_lse: bool = True, want_flags: bool = False,
                         out=None, workspace=None, stream=None):
    """Causal attention of each sequence's chunk q [total, heads, head_dim]
    (bfloat16 or float16, any token and head strides) over its pages; the chunk's
    own keys and values must be in the cache (spec_kv_append).  scale defaults to
    head_dim^-1/2; window w > 0 shows a query only its last w keys (0: all; no
    sequence reaches 2^31 of them).  Returns a dict:
    out [total, heads, head_dim], lse [total, heads] float32 (if want_lse),
    flags [B] uint8 (if want_flags)."""
    torch = _torch()
    L = _lib or load()
    _check_rows(q, 0, cache, "q")
    B = _check_index(block_table, q_start, kv_len, cache.device)
    total, heads, dim = q.shape
    window = max(-1, min(int(window), 2**31 - 1))  # (the library refuses what is negative)
    dev = q.device
    o = dict(out or {})
    _output(o, "out", (total, heads, dim), q.dtype, dev, stream)
    _output(o, "lse", (total, heads), torch.float32, dev, stream, want_lse)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags)
    sh = _stream_of(stream, dev)
    need = attention_workspace_bytes(cache, heads)
    ws = _workspace(workspace, need, dev, sh, stream)
    batch = _BatchStruct(block_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(), total, B,
                         block_table.shape[1])
    rc = _queue(L.spec_chunk_attention, dev, cache._ref, ctypes.addressof(batch), _address(q),
                _row_code(q), heads, q.stride(0), q.stride(1),
                dim ** -0.5 if scale is None else float(scale), window, _address(o["out"]),
                _address(o.get("lse")), _address(o.get("flags")), _address(ws), ws.numel(), sh)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_chunk_attention")
    return o


def spec_verify_probs(target_probs, draft_probs, draft_tokens, uniforms, *,
                      want_flags: bool = False, out=None, stream=None):
    """The round from given probabilities (float32 or bfloat16) and given uniforms
    [B, gamma+1] float32 (the accept tests', then the draw's).  Returns a dict:
    tokens [B, g+1] int32, counts [B] int32, flags [B] uint8 (if want_flags)."""
    torch = _torch()
    L = _lib or load()
    B, g1, V = target_probs.shape
    g = g1 - 1
    if tuple(draft_probs.shape) != (B, g, V) or tuple(draft_tokens.shape) != (B, g) or \
            tuple(uniforms.shape) != (B, g1):
        raise ValueError("shape mismatch: target [B,g+1,V], draft [B,g,V], tokens [B,g], "
                         "uniforms [B,g+1]")
    if draft_probs.dtype != target_probs.dtype or draft_tokens.dtype != torch.int32 or \
            uniforms.dtype != torch.float32:
        raise TypeError("draft probs must match target dtype; draft tokens must be int32, "
                        "uniforms float32")
    _check_cuda(target_probs, draft_probs, draft_tokens, uniforms)
    dev = target_probs.device
    o = dict(out or {})
    _output(o, "tokens", (B, g1), torch.int32, dev, stream)
    _output(o, "counts", (B,), torch.int32, dev, stream)
    _output(o, "flags", (B,), torch.uint8, dev, stream, want_flags)
    rc = _queue(L.spec_verify_probs, dev, _address(target_probs), _address(draft_probs),
                _address(draft_tokens), _address(uniforms), B, g, V, _dtype_code(target_probs),
                _address(o["tokens"]), _address(o["counts"]), _address(o.get("flags")),
                _stream_of(stream, dev))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_probs")
    return o
