"""Batched speculative-decoding verification on GB300 (sm_103a).

Python binding of ``libspecverify.so`` (C ABI in ``include/specverify.h``).
This module only marshals arguments: torch CUDA tensors are checked for
dtype, device and layout and their pointers, strides and the current CUDA
stream are passed to the library, whose kernels do every step of the
verification (for append_kv, read_kv, paged_attention and warp_sample a small C++
extension does so, ``csrc/tensors.cpp``).  There is no CPU path: if the library is missing or a tensor is
not on a CUDA device, the call raises.

The operation is the one on the "spec-verify" page (Hugging Face kernels page
phanerozoic/spec-verify), section "Usage":
``n_accepted, next_token = verify_greedy(target_probs, draft_tokens)`` -- keep
``draft_tokens[:n_accepted]`` and append ``next_token`` -- batched over B
sequences, plus the speculative-sampling rule of section "Method".
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from . import _build
from . import trace as _trace
from .trace import TRACE_EVENTS

LIBRARY = _build.LIBRARY

SV_OK = 0
SV_EINVAL = -1
SV_EWORKSPACE = -2
SV_ECUDA = -3
SV_ETOOLARGE = -4
NOALLOC_SCRATCH_BYTES = 4 << 20
STATUS_BAD_TOKEN = 1
STATUS_ZERO_MASS = 2
STATUS_OVERFLOW = 4
STATUS_BAD_MODE = 8
STATUS_TIMEOUT = 16
STATUS_BAD_VALUE = 32   # verification: debug builds only (built with SV_DEBUG=1); warp_sample: always
STATUS_BAD_PAGE = 64
STATUS_BAD_LENGTH = 128
MAX_K = 64

# every symbol include/specverify.h declares
EXPORTED = (
    "sv_workspace_size", "sv_workspace_init", "sv_verify_greedy", "sv_verify_sample",
    "sv_verify_round", "sv_get_status", "sv_set_ctas_per_sm", "sv_last_grid_size",
    "sv_last_kernel_count", "sv_alpha", "sv_verify_sample_logits",
    "sv_status_string", "sv_version", "sv_verify_sample_noalloc", "sv_trace_reset",
    "sv_trace_read", "sv_cache_workspace_size", "sv_append_kv", "sv_paged_attention",
    "sv_warp_sample", "sv_append_kv_normed", "sv_read_kv", "sv_paged_attention_scaled",
    "sv_paged_attention_scratch_size",
)

_lock = threading.Lock()
_lib = None


class SpecVerifyError(RuntimeError):
    pass


def build(force: bool = False) -> str:
    """Compiles libspecverify.so in-tree (nvcc, sm_103a) and the extension
    beside it."""
    return _build.build(force=force)


def load():
    """The ctypes handle of libspecverify.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIBRARY):
            raise SpecVerifyError(
                f"{LIBRARY} is missing: build it with "
                "speculative_decoding_verification_08_gb300.build() (no CPU fallback exists)")
        _lib = _declare(ctypes.CDLL(LIBRARY))
        return _lib


def _declare(lib):
    """Sets the argument and result types of every C-ABI call on a loaded
    copy of the library (the regular build, or a debug build)."""
    P = ctypes.c_void_p
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.sv_workspace_size.argtypes = [i32, i32, i64]
    lib.sv_workspace_size.restype = sz
    lib.sv_workspace_init.argtypes = [P, sz, P]
    lib.sv_workspace_init.restype = ctypes.c_int
    lib.sv_verify_greedy.argtypes = [P, i64, P, i32, i32, i64, P, P, P, sz, P]
    lib.sv_verify_greedy.restype = ctypes.c_int
    lib.sv_verify_sample.argtypes = [P, i64, P, i64, P, P, P, i32, i32, i64, P, P, P, sz, P]
    lib.sv_verify_sample.restype = ctypes.c_int
    lib.sv_verify_round.argtypes = [P, P, i64, P, i64, P, P, P, i32, i32, i64, P, P,
                                    P, P, i32, P, sz, P]
    lib.sv_verify_round.restype = ctypes.c_int
    lib.sv_get_status.argtypes = [P, P, P]
    lib.sv_get_status.restype = ctypes.c_int
    lib.sv_set_ctas_per_sm.argtypes = [i32]
    lib.sv_set_ctas_per_sm.restype = ctypes.c_int
    lib.sv_last_grid_size.argtypes = []
    lib.sv_last_grid_size.restype = i64
    lib.sv_last_kernel_count.argtypes = []
    lib.sv_last_kernel_count.restype = i32
    lib.sv_alpha.argtypes = [P, i64, P, i64, i32, i32, i64, P, P, P, sz, P]
    lib.sv_alpha.restype = ctypes.c_int
    lib.sv_verify_sample_logits.argtypes = [P, i64, P, i64, P, P, P, i32, i32, i64,
                                            ctypes.c_float, P, P, P, sz, P]
    lib.sv_verify_sample_logits.restype = ctypes.c_int
    lib.sv_status_string.argtypes = [ctypes.c_int]
    lib.sv_status_string.restype = ctypes.c_char_p
    lib.sv_version.argtypes = []
    lib.sv_version.restype = ctypes.c_int
    lib.sv_verify_sample_noalloc.argtypes = [P, i64, P, i64, P, P, P, i32, i32, i64, P, P, P]
    lib.sv_verify_sample_noalloc.restype = ctypes.c_int
    lib.sv_trace_reset.argtypes = [P]
    lib.sv_trace_reset.restype = ctypes.c_int
    lib.sv_trace_read.argtypes = [P, sz, ctypes.POINTER(sz), P]
    lib.sv_trace_read.restype = ctypes.c_int
    C = S = ctypes.c_char_p      # sv_paged_cache and strides, packed
    lib.sv_cache_workspace_size.argtypes = []
    lib.sv_cache_workspace_size.restype = sz
    lib.sv_append_kv.argtypes = [C, P, S, P, S, P, S, P, S, i32, P, i32, i32, P, P, sz, P]
    lib.sv_append_kv.restype = ctypes.c_int
    lib.sv_paged_attention.argtypes = [C, P, S, P, S, i32, ctypes.c_float, i32, P, sz, P]
    lib.sv_paged_attention.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.sv_append_kv_normed.argtypes = [C, C, i32, P, S, P, S, P, S, P, S, i32, P, P, i32, f32, P, i32, i32, P, P,
                                        sz, P]
    lib.sv_append_kv_normed.restype = ctypes.c_int
    lib.sv_read_kv.argtypes = [C, C, i32, P, S, P, S, P, sz, P]
    lib.sv_read_kv.restype = ctypes.c_int
    lib.sv_paged_attention_scratch_size.argtypes = [C, i32]
    lib.sv_paged_attention_scratch_size.restype = sz
    lib.sv_paged_attention_scaled.argtypes = [C, C, i32, P, S, P, S, i32, f32, i32, P, sz, P, sz, P]
    lib.sv_paged_attention_scaled.restype = ctypes.c_int
    lib.sv_warp_sample.argtypes = [P, i64, i32, i32, i64, P, P, P, P, P, P, P, i64, P, sz, P]
    lib.sv_warp_sample.restype = ctypes.c_int
    return lib


def status_string(code: int) -> str:
    return load().sv_status_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc != SV_OK:
        raise SpecVerifyError(f"{what}: {status_string(rc)} (code {rc})")


def workspace_size(B: int, K: int, V: int) -> int:
    return int(load().sv_workspace_size(B, K, V))


def set_ctas_per_sm(n: int):
    """Persistent-grid residency override (0 = as many CTAs as the SMs hold)."""
    _check(load().sv_set_ctas_per_sm(int(n)), "sv_set_ctas_per_sm")


def last_grid_size() -> int:
    return int(load().sv_last_grid_size())


def last_kernel_count() -> int:
    """Kernels the last verification call on this thread enqueued."""
    return int(load().sv_last_kernel_count())


def _torch():
    import torch
    return torch


def _stream_handle(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Workspace:
    """Device scratch for B sequences, K drafts and vocabulary V (zeroed once)."""

    def __init__(self, B: int, K: int, V: int, device=None, stream=None):
        torch = _torch()
        nbytes = workspace_size(B, K, V)
        if nbytes == 0:
            raise SpecVerifyError(f"invalid sizes B={B} K={K} V={V}")
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.B, self.K, self.V, self.nbytes = B, K, V, nbytes
        _check(load().sv_workspace_init(self.ptr, nbytes, _stream_handle(stream)),
               "sv_workspace_init")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    def fits(self, B, K, V) -> bool:
        return workspace_size(B, K, V) <= self.nbytes

    def status(self, stream=None) -> int:
        """Waits for the stream and returns (and clears) the device status bits."""
        out = ctypes.c_uint32(0)
        _check(load().sv_get_status(self.ptr, _stream_handle(stream), ctypes.byref(out)),
               "sv_get_status")
        return int(out.value)


_ws_cache = {}


def _workspace(ws, B, K, V, device, stream=None):
    """The caller's workspace, or one kept for these sizes and this stream.
    Calls that share a workspace must be ordered on one stream, so calls on
    different streams never share an implicit one."""
    if ws is not None:
        if not ws.fits(B, K, V):
            raise SpecVerifyError("workspace too small for these sizes")
        return ws
    key = (str(device), B, K, V, _stream_handle(stream).value)
    w = _ws_cache.get(key)
    if w is None:
        w = Workspace(B, K, V, device, stream)
        _ws_cache[key] = w
    return w


def _device_of(x):
    """The CUDA device a call on x runs on: x's own, or the current one for a
    pinned CPU tensor."""
    torch = _torch()
    return x.device if x.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _usable(x) -> bool:
    """A CUDA tensor, or a CPU tensor in page-locked memory (read in place)."""
    return x.is_cuda or x.is_pinned()


def _rows3(x, rows, name, dtype):
    """(tensor viewed as [B][rows][V], B, V, row stride) with the library's layout."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or not _usable(x):
        raise SpecVerifyError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
    if x.dtype != dtype:
        raise SpecVerifyError(f"{name} must be {dtype}, got {x.dtype}")
    if x.dim() == 2:
        x = x.unsqueeze(0)
    if x.dim() != 3 or x.shape[1] != rows:
        raise SpecVerifyError(f"{name}: expected [B][{rows}][V], got {tuple(x.shape)}")
    B, _, V = x.shape
    if x.stride(2) != 1:
        raise SpecVerifyError(f"{name}: the vocabulary dimension must be contiguous")
    rs = x.stride(1) if rows > 1 else (x.stride(0) if B > 1 else V)
    if rows > 1 and B > 1 and x.stride(0) != rows * rs:
        raise SpecVerifyError(f"{name}: rows of all sequences must be evenly strided")
    if rs < V:
        raise SpecVerifyError(f"{name}: row stride {rs} < V={V}")
    return x, B, V, rs


def _vec(x, n, name, dtype, device):
    torch = _torch()
    if x is None:
        return None
    if not isinstance(x, torch.Tensor) or not (x.is_pinned() or (x.is_cuda and x.device == device)):
        raise SpecVerifyError(f"{name} must be a CUDA tensor on {device} or a pinned CPU tensor")
    if x.dtype != dtype:
        raise SpecVerifyError(f"{name} must be {dtype}, got {x.dtype}")
    if not x.is_contiguous() or x.numel() != n:
        raise SpecVerifyError(f"{name}: expected {n} contiguous elements")
    return x


def _ptr(x):
    return ctypes.c_void_p(0 if x is None else x.data_ptr())


def _outputs(B, device, n_out, next_out):
    torch = _torch()
    if n_out is None:
        n_out = torch.empty(B, dtype=torch.int32, device=device)
    if next_out is None:
        next_out = torch.empty(B, dtype=torch.int32, device=device)
    _vec(n_out, B, "n_accepted", torch.int32, device)
    _vec(next_out, B, "next_token", torch.int32, device)
    return n_out, next_out


def verify_greedy(p, t, *, ws=None, n_out=None, next_out=None, stream=None):
    """Greedy verification.  p: [B][K+1][V] (or [K+1][V]) f32, t: [B][K] (or [K])
    int32 -> (n_accepted [B] int32, next_token [B] int32) on the same device."""
    torch = _torch()
    K = t.shape[-1]
    p, B, V, ps = _rows3(p, K + 1, "p", torch.float32)
    dev = _device_of(p)
    t = _vec(t, B * K, "t", torch.int32, dev)
    n_out, next_out = _outputs(B, dev, n_out, next_out)
    w = _workspace(ws, B, K, V, dev, stream)
    rc = load().sv_verify_greedy(_ptr(p), ps, _ptr(t), B, K, V, _ptr(n_out), _ptr(next_out),
                                 w.ptr, w.nbytes, _stream_handle(stream))
    _check(rc, "sv_verify_greedy")
    return n_out, next_out


def verify_sample(p, q, t, u_acc, u_res, *, ws=None, n_out=None, next_out=None, stream=None):
    """Speculative-sampling verification.  p: [B][K+1][V] f32, q: [B][K][V] f32,
    t: [B][K] int32, u_acc: [B][K] f32, u_res: [B] f64 -> (n_accepted, next_token)."""
    torch = _torch()
    K = t.shape[-1]
    p, B, V, ps = _rows3(p, K + 1, "p", torch.float32)
    dev = _device_of(p)
    q, Bq, Vq, qs = _rows3(q, K, "q", torch.float32) if K > 0 else (None, B, V, V)
    if (Bq, Vq) != (B, V):
        raise SpecVerifyError("q does not match p")
    t = _vec(t, B * K, "t", torch.int32, dev)
    u_acc = _vec(u_acc, B * K, "u_acc", torch.float32, dev)
    u_res = _vec(u_res, B, "u_res", torch.float64, dev)
    n_out, next_out = _outputs(B, dev, n_out, next_out)
    w = _workspace(ws, B, K, V, dev, stream)
    rc = load().sv_verify_sample(_ptr(p), ps, _ptr(q), qs, _ptr(t), _ptr(u_acc), _ptr(u_res),
                                 B, K, V, _ptr(n_out), _ptr(next_out), w.ptr, w.nbytes,
                                 _stream_handle(stream))
    _check(rc, "sv_verify_sample")
    return n_out, next_out


def verify_sample_noalloc(p, q, t, u_acc, u_res, *, n_out=None, next_out=None, stream=None):
    """verify_sample without a workspace, for callers that cannot allocate
    device memory while enqueueing work (framework hooks or plugin interfaces
    that forbid allocation, serving loops that must not risk a synchronising
    or failing cudaMalloc).  The scratch is a fixed 4 MiB array inside the
    library; larger sizes raise (SV_ETOOLARGE).  Calls share that array, so
    calls that overlap on the GPU race.  Pass n_out/next_out to avoid the two
    output allocations this wrapper would otherwise make."""
    torch = _torch()
    K = t.shape[-1]
    p, B, V, ps = _rows3(p, K + 1, "p", torch.float32)
    dev = _device_of(p)
    q, Bq, Vq, qs = _rows3(q, K, "q", torch.float32) if K > 0 else (None, B, V, V)
    if (Bq, Vq) != (B, V):
        raise SpecVerifyError("q does not match p")
    t = _vec(t, B * K, "t", torch.int32, dev)
    u_acc = _vec(u_acc, B * K, "u_acc", torch.float32, dev)
    u_res = _vec(u_res, B, "u_res", torch.float64, dev)
    n_out, next_out = _outputs(B, dev, n_out, next_out)
    rc = load().sv_verify_sample_noalloc(_ptr(p), ps, _ptr(q), qs, _ptr(t), _ptr(u_acc),
                                         _ptr(u_res), B, K, V, _ptr(n_out), _ptr(next_out),
                                         _stream_handle(stream))
    _check(rc, "sv_verify_sample_noalloc")
    return n_out, next_out


def verify_sample_logits(zp, zq, t, u_acc, u_res, temperature: float = 1.0, *, ws=None,
                         n_out=None, next_out=None, stream=None):
    """Sampling verification from logits: zp [B][K+1][V], zq [B][K][V] f32 (or
    [K+1][V] / [K][V]), warped by softmax(z / temperature) on the fly ->
    (n_accepted, next_token) int32 [B]."""
    torch = _torch()
    t_ = t if t.dim() == 2 else t.reshape(1, -1)
    K = t_.shape[1]
    zp, B, V, ps = _rows3(zp, K + 1, "zp", torch.float32)
    dev = _device_of(zp)
    zq, Bq, Vq, qs = _rows3(zq, K, "zq", torch.float32) if K > 0 else (None, B, V, V)
    if K > 0 and (Bq, Vq) != (B, V):
        raise SpecVerifyError("zq shape does not match zp")
    t = _vec(t, B * K, "t", torch.int32, dev)
    u_acc = _vec(u_acc, B * K, "u_acc", torch.float32, dev)
    u_res = _vec(u_res, B, "u_res", torch.float64, dev)
    n_out, next_out = _outputs(B, dev, n_out, next_out)
    w = _workspace(ws, B, K, V, dev, stream)
    _check(load().sv_verify_sample_logits(_ptr(zp), ps, _ptr(zq), qs, _ptr(t), _ptr(u_acc),
                                          _ptr(u_res), B, K, V, float(temperature), _ptr(n_out),
                                          _ptr(next_out), w.ptr, w.nbytes,
                                          _stream_handle(stream)),
           "sv_verify_sample_logits")
    return n_out, next_out


def alpha(p, q, *, ws=None, alpha_out=None, expected_out=None, stream=None):
    """Acceptance-rate diagnostic: p [B][K+1][V], q [B][K][V] f32 ->
    (alpha [B][K] f64, expected accepted length [B] f64), with
    alpha[b][i] = sum_v min(p_i / P_i, q_i / Q_i) over row totals P_i, Q_i."""
    torch = _torch()
    q3, B, V, qs = _rows3(q, q.shape[-2] if q.dim() >= 2 else 1, "q", torch.float32)
    K = q3.shape[1]
    p, Bp, Vp, ps = _rows3(p, K + 1, "p", torch.float32)
    if (Bp, Vp) != (B, V):
        raise SpecVerifyError("q shape does not match p")
    dev = _device_of(p)
    if alpha_out is None:
        alpha_out = torch.empty(B, K, dtype=torch.float64, device=dev)
    if expected_out is None:
        expected_out = torch.empty(B, dtype=torch.float64, device=dev)
    _vec(alpha_out.reshape(-1), B * K, "alpha_out", torch.float64, dev)
    _vec(expected_out, B, "expected_out", torch.float64, dev)
    w = _workspace(ws, B, K, V, dev, stream)
    _check(load().sv_alpha(_ptr(p), ps, _ptr(q3), qs, B, K, V, _ptr(alpha_out),
                           _ptr(expected_out), w.ptr, w.nbytes, _stream_handle(stream)),
           "sv_alpha")
    return alpha_out, expected_out


def verify_round(mode, p, q, t, u_acc, u_res, *, tokens=None, lengths=None, ws=None,
                 n_out=None, next_out=None, stream=None):
    """Mixed round: mode [B] uint8 (0 greedy, 1 sampling) picks each sequence's
    rule.  With tokens [B][max_len] int32 and lengths [B] int32 the round is
    committed in place (t[b][:n] then next appended)."""
    torch = _torch()
    K = t.shape[-1]
    p, B, V, ps = _rows3(p, K + 1, "p", torch.float32)
    dev = _device_of(p)
    q, Bq, Vq, qs = _rows3(q, K, "q", torch.float32) if K > 0 else (None, B, V, V)
    if (Bq, Vq) != (B, V):
        raise SpecVerifyError("q does not match p")
    mode = _vec(mode, B, "mode", torch.uint8, dev)
    t = _vec(t, B * K, "t", torch.int32, dev)
    u_acc = _vec(u_acc, B * K, "u_acc", torch.float32, dev)
    u_res = _vec(u_res, B, "u_res", torch.float64, dev)
    max_len = 0
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise SpecVerifyError("tokens must be [B][max_len]")
        max_len = tokens.shape[1]
        _vec(tokens, B * max_len, "tokens", torch.int32, dev)
        _vec(lengths, B, "lengths", torch.int32, dev)
    n_out, next_out = _outputs(B, dev, n_out, next_out)
    w = _workspace(ws, B, K, V, dev, stream)
    rc = load().sv_verify_round(_ptr(mode), _ptr(p), ps, _ptr(q), qs, _ptr(t), _ptr(u_acc),
                                _ptr(u_res), B, K, V, _ptr(n_out), _ptr(next_out), _ptr(tokens),
                                _ptr(lengths), max_len, w.ptr, w.nbytes, _stream_handle(stream))
    _check(rc, "sv_verify_round")
    return n_out, next_out


class HostVerifier:
    """Verification of host-resident inputs through the public calls.  Inputs
    are pinned CPU tensors; (n_accepted, next_token) come back in pinned
    memory and each call waits for them.

    mapped=True (default): the inputs are handed to the library where they
    are; the kernels read them over the host link, and only the rows the rule
    needs (the residual pair or bonus row of a sampling sequence, the rows up
    to the first miss of a greedy one) cross it.  mapped=False: every call
    first copies all inputs into device buffers."""

    def __init__(self, B: int, K: int, V: int, device=None, sampling: bool = True,
                 mapped: bool = True):
        torch = _torch()
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.B, self.K, self.V, self.device, self.mapped = B, K, V, dev, mapped
        self.sampling = sampling
        if not mapped:
            self.p = torch.empty(B, K + 1, V, dtype=torch.float32, device=dev)
            self.q = torch.empty(B, K, V, dtype=torch.float32, device=dev) if sampling else None
            self.t = torch.empty(B, K, dtype=torch.int32, device=dev)
            self.u_acc = torch.empty(B, K, dtype=torch.float32, device=dev)
            self.u_res = torch.empty(B, dtype=torch.float64, device=dev)
        self.n = torch.empty(B, dtype=torch.int32, device=dev)
        self.next = torch.empty(B, dtype=torch.int32, device=dev)
        self.n_host = torch.empty(B, dtype=torch.int32, pin_memory=True)
        self.next_host = torch.empty(B, dtype=torch.int32, pin_memory=True)
        self.ws = Workspace(B, K, V, dev)

    def h2d_bytes(self) -> int:
        """Bytes of input that crossed the host link in the last call: all of
        them when copying, else what the rule read (from its n_accepted)."""
        B, K, V = self.B, self.K, self.V
        if not self.mapped:
            n = (K + 1) * V * 4 * B + K * 4 * B
            if self.sampling:
                n += K * V * 4 * B + K * 4 * B + 8 * B
            return n
        total = 0
        for n in self.n_host.tolist():
            if self.sampling:
                rows = 8 * V if n < K else 4 * V
                total += rows + 64 * min(n + 1, K) + 8 * K + 8
            else:
                total += (n + 1) * 4 * V + 4 * K + 4 * min(n + 1, K)
        return total

    def d2h_bytes(self) -> int:
        return self.B * 8

    def _pinned(self, *xs):
        for x in xs:
            if x is not None and not x.is_pinned():
                raise SpecVerifyError("HostVerifier inputs must be pinned CPU tensors")

    def sample(self, p, q, t, u_acc, u_res):
        self._pinned(p, q, t, u_acc, u_res)
        if not self.mapped:
            self.p.copy_(p, non_blocking=True)
            self.q.copy_(q, non_blocking=True)
            self.t.copy_(t, non_blocking=True)
            self.u_acc.copy_(u_acc, non_blocking=True)
            self.u_res.copy_(u_res, non_blocking=True)
            p, q, t, u_acc, u_res = self.p, self.q, self.t, self.u_acc, self.u_res
        verify_sample(p, q, t, u_acc, u_res, ws=self.ws, n_out=self.n, next_out=self.next)
        return self._finish()

    def greedy(self, p, t):
        self._pinned(p, t)
        if not self.mapped:
            self.p.copy_(p, non_blocking=True)
            self.t.copy_(t, non_blocking=True)
            p, t = self.p, self.t
        verify_greedy(p, t, ws=self.ws, n_out=self.n, next_out=self.next)
        return self._finish()

    def _finish(self):
        torch = _torch()
        self.n_host.copy_(self.n, non_blocking=True)
        self.next_host.copy_(self.next, non_blocking=True)
        torch.cuda.current_stream().synchronize()
        return self.n_host, self.next_host


# ---------------------------------------------------------------------------
# the target pass of a round: paged cache, attention over it, warped rows

class CacheWorkspace:
    """Device scratch of append_kv, paged_attention and warp_sample: one size
    for all sizes, one call at a time in stream order."""

    def __init__(self, device=None, stream=None):
        torch = _torch()
        self.nbytes = int(load().sv_cache_workspace_size())
        dev = _cuda_index(device, stream)
        # (from the pool of the stream it serves: what another stream still has
        # to do with a freed block must not land in it)
        with torch.cuda.device(dev), _on(stream):
            _no_capture("is zeroed once, when it is made: make it before the capture")
            self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
            self.ptr = self.buf.data_ptr()
            self.reset(stream)

    def reset(self, stream=None):
        """Zeroes the workspace, in stream order."""
        with _torch().cuda.device(self.buf.device):
            _check(load().sv_workspace_init(self.ptr, self.nbytes, _stream_handle(stream)),
                   "sv_workspace_init")

    def status(self, stream=None) -> int:
        """Waits for the stream and returns (and clears) the device status bits.
        After STATUS_TIMEOUT or STATUS_OVERFLOW the workspace is zeroed as well:
        counts that a call did not finish are left in it."""
        out = ctypes.c_uint32(0)
        with _torch().cuda.device(self.buf.device):
            _check(load().sv_get_status(self.ptr, _stream_handle(stream), ctypes.byref(out)),
                   "sv_get_status")
        if out.value & (STATUS_TIMEOUT | STATUS_OVERFLOW):
            self.reset(stream)
        return int(out.value)


def _on(stream):
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _cuda_index(device, stream) -> int:
    """The device meant: the one named, else the stream's, else the current one."""
    torch = _torch()
    index = None
    if device is not None:
        named = torch.device(device)
        if named.type != "cuda":
            raise SpecVerifyError(f"a CacheWorkspace lives on a CUDA device, not on {named}")
        index = named.index
    if index is None and stream is not None:
        index = stream.device.index
    return torch.cuda.current_device() if index is None else index


def _no_capture(what):
    if _torch_c()._cuda_isCurrentStreamCapturing():
        raise SpecVerifyError(f"a CacheWorkspace {what}")


def cache_workspace(device=None, stream=None) -> CacheWorkspace:
    """The workspace that calls without one share on this device and stream
    (calls on different streams never share an implicit one, and a call that is
    captured into a graph has none)."""
    dev = _cuda_index(device, stream)
    return _cache_ws(None, dev, _raw_stream(dev, stream), stream)


def _raw_stream(device, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    # (the plain handle: a Stream object costs more than the rest of the checks)
    return _torch_c()._cuda_getCurrentRawStream(device)


_TORCH_C = None


def _torch_c():
    global _TORCH_C
    if _TORCH_C is None:
        _TORCH_C = _torch()._C
    return _TORCH_C


def _cache_ws(ws, device, raw, stream):
    if ws is not None:
        return ws
    # (a graph keeps the workspace's address and may be replayed on any stream,
    # beside other graphs)
    _no_capture("of its own is needed by a captured call: pass ws=, made before the capture")
    key = (device, raw)
    w = _ws_cache.get(key)
    if w is None:
        w = _ws_cache[key] = CacheWorkspace(_torch().device("cuda", device), stream)
    return w


_tensors = None


def _native():
    """The extension that checks the tensors of these calls and hands them to
    the library."""
    global _tensors
    lib = load()
    with _lock:
        if _tensors is None:
            _torch()
            if not os.path.exists(_build.EXTENSION):
                raise SpecVerifyError(f"{_build.EXTENSION} is missing: build it with "
                                      "speculative_decoding_verification_08_gb300.build()")
            loader = importlib.machinery.ExtensionFileLoader(__name__ + "._tensors", _build.EXTENSION)
            spec = importlib.util.spec_from_file_location(loader.name, _build.EXTENSION, loader=loader)
            module = importlib.util.module_from_spec(spec)
            loader.exec_module(module)
            def at(*calls):
                return (ctypes.cast(f, ctypes.c_void_p).value for f in calls)
            module.bind(*at(lib.sv_append_kv, lib.sv_paged_attention, lib.sv_warp_sample),
                        SpecVerifyError, _check)
            module.bind8(*at(lib.sv_append_kv_normed, lib.sv_read_kv, lib.sv_paged_attention_scaled,
                             lib.sv_paged_attention_scratch_size))
            _tensors = module
        return _tensors


def _call(name, x, what, args, ws, stream):
    """One call on x's device and, unless one is given, its current stream.  On a
    stream other than the current one the outputs come from that stream's pool,
    as if it were current."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return _call(name, x, what, args, ws, None)
    device = x.get_device()
    if device < 0:
        raise SpecVerifyError(f"{what} must be a CUDA tensor")
    raw = _raw_stream(device, None)
    w = _cache_ws(ws, device, raw, None)
    return getattr(_tensors or _native(), name)(*args, w.ptr, w.nbytes, raw)


def append_kv(k, v, k_cache, v_cache, pages, q_start, kv_len, *, inv_freq=None, q=None,
              q_out=None, positions=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
              k_scale=None, v_scale=None, ws=None, stream=None):
    """Writes the new tokens' keys and values [N][kv_heads][D] into their slots
    of the paged cache [pages][page_size][kv_heads][D] (any order of the axes),
    the keys rotated by their positions, and returns q [N][q_heads][D] rotated
    alike (None without q; q_out may be q itself).

    pages [B][max_pages] int32, q_start [B + 1] int32 (rows of each sequence's
    new tokens), kv_len [B] int32 (lengths with the new tokens).  inv_freq
    [rot_dim / 2] f64 gives radians per position of each pair (None: no
    rotation); pairs are (i, i + rot_dim / 2), or (2i, 2i + 1) when
    interleaved.  positions [N] int32 overrides the slots as positions.

    q_norm, k_norm [D] (f32 or the tokens' type) norm each head before it
    turns: x / sqrt(mean(x^2) + eps) * norm.  With k_scale and v_scale
    [pages][page_size][kv_heads] (float8_e8m0fnu, any order of the axes) the
    caches are float8_e4m3fn: each vector is divided by the power of two that
    brings its largest magnitude to 448 or less, and rounded once."""
    if q_norm is None and k_norm is None and k_scale is None and v_scale is None:
        return _call("append_kv", k_cache, "k_cache",
                     (k, v, k_cache, v_cache, pages, q_start, kv_len, inv_freq, q, q_out, positions, interleaved),
                     ws, stream)
    return _call("append_kv_normed", k_cache, "k_cache",
                 (k, v, k_cache, v_cache, pages, q_start, kv_len, inv_freq, q, q_out, positions, interleaved,
                  q_norm, k_norm, eps, k_scale, v_scale), ws, stream)


def read_kv(k_cache, v_cache, pages, q_start, kv_len, *, rows=None, dtype=None, k_scale=None, v_scale=None,
            k_out=None, v_out=None, ws=None, stream=None):
    """The way back from a paged cache: (k, v) [rows][kv_heads][D], row
    q_start[b] + j of n being what slot kv_len[b] - n + j holds, as append_kv
    put it there (n = kv_len[b] for whole sequences).  `rows` says how many
    there are in all (q_start's last entry, which only the device knows) unless
    k_out or v_out does.  A float8_e4m3fn cache (k_scale and v_scale as for
    append_kv) comes back as `dtype`, bfloat16 or float16 (default bfloat16),
    others as what they are."""
    code = 0
    if dtype is not None or k_scale is not None:
        torch = _torch()
        code = {None: 1, torch.bfloat16: 1, torch.float16: 2}.get(dtype)
        if code is None:
            raise SpecVerifyError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    return _call("read_kv", k_cache, "k_cache",
                 (k_cache, v_cache, pages, q_start, kv_len, -1 if rows is None else rows, code, k_scale, v_scale,
                  k_out, v_out), ws, stream)


def paged_attention(q, k_cache, v_cache, pages, q_start, kv_len, *, scale=None, window=0,
                    out=None, k_scale=None, v_scale=None, ws=None, stream=None):
    """Attention of the new tokens q [N][q_heads][D] over the paged cache that
    holds them already (append_kv): causal, over the last `window` slots when
    window > 0, scale 1 / sqrt(D) by default; q_heads a multiple of kv_heads.
    Arrays as for append_kv; a float8_e4m3fn cache comes with its k_scale and
    v_scale.  Rows that see nothing are zeros.  Returns out
    [N][q_heads][D].

    Over an 8-bit cache whose sequences have many new tokens (more than 128 rows,
    tokens times q_heads / kv_heads, on the batch's average) the call first reads
    them back to 16 bits, into memory of its own from the current stream's pool:
    four bytes for each key and value pair of the table's pages or of the cache's,
    whichever are fewer.  Where that much cannot be had, or the table's slots
    would be more than 16 GiB so, it attends to the codes all the same (slower
    for such batches).  What differs by the way taken, besides roundings: keys
    and values of float16 tokens past 65504, which the codes hold, saturate when
    they are read back, and scores past 2^26 may then give NaN.  Vectors that are
    NaN reach the rows that see them and no others, either way.  A long chunk
    beside many short rounds does better in a call of its own."""
    if k_scale is None and v_scale is None:
        return _call("paged_attention", k_cache, "k_cache",
                     (q, k_cache, v_cache, pages, q_start, kv_len, scale, window, out), ws, stream)
    return _call("paged_attention_scaled", k_cache, "k_cache",
                 (q, k_cache, v_cache, pages, q_start, kv_len, scale, window, out, k_scale, v_scale), ws, stream)


def warp_sample(z, u=None, *, temperature=None, top_k=None, top_p=None, min_p=None, probs=False,
                probs_out=None, token_out=None, ws=None, stream=None):
    """Warps rows of logits z [..., V] (f32, bf16 or f16) by temperature, top-k,
    top-p and min-p, in this order, each on what the one before left, and draws
    a token per row with u [...] f64 in [0, 1).  The filters are tensors with
    one value per row (f32; top_k int32) or None (off).  Returns (token int32
    or None without u, probs [..., V] f32 or None unless probs or probs_out):
    rows as verify_sample takes them; probs_out must not overlap z.  A row
    without mass or with a NaN or +inf logit gives token -1 and zeros."""
    return _call("warp_sample", z, "z",
                 (z, u, temperature, top_k, top_p, min_p, probs, probs_out, token_out), ws, stream)


# ---------------------------------------------------------------------------
# timeline of the item kernel (a library built with SV_TRACE=1)

TRACE_RECORDS = 2048 * 1024


def trace_reset(stream=None, lib=None):
    """Clears the trace buffer on the stream (a trace build; SpecVerifyError otherwise)."""
    _check((lib or load()).sv_trace_reset(_stream_handle(stream)), "sv_trace_reset")


def trace_read(stream=None, lib=None):
    """The recorded events as a uint64 array [N][2] (time in ns, event word),
    empty slots dropped; waits for the stream."""
    import numpy as np
    buf = np.zeros((TRACE_RECORDS, 2), dtype=np.uint64)
    n = ctypes.c_size_t(0)
    _check((lib or load()).sv_trace_read(buf.ctypes.data_as(ctypes.c_void_p), TRACE_RECORDS,
                                         ctypes.byref(n), _stream_handle(stream)),
           "sv_trace_read")
    buf = buf[:n.value]
    return buf[buf[:, 0] != 0]


def trace_summary(records) -> dict:
    """Where one traced launch's time went (``trace.summary``)."""
    return _trace.summary(records)


def trace_timeline(records) -> dict:
    """Per-launch summaries of several consecutive traced launches and the
    time between them (``trace.timeline``)."""
    return _trace.timeline(records)
