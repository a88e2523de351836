"""Thin Python binding of libdspark.so (ctypes; argument marshalling only).

Every function takes CUDA torch tensors, passes their device pointers and the
current CUDA stream, or the one given as ``stream``, to the C ABI of
``include/dspark.h`` and returns the output tensors it allocated (on the stream
that writes them).  All arithmetic of the cycle runs in the
library's kernels; this module only checks types, allocates outputs and the
workspace, and translates status codes into exceptions.  There is no CPU
fallback: if the library cannot be loaded, importing a function raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import _build

F32 = 0
BF16 = 1
E4M3 = 2

_lock = threading.Lock()
_lib = None

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported dtype", -3: "unsupported sizes",
          -4: "CUDA runtime error", -5: "bounded device wait ran out", -6: "token id outside [0, V)",
          -7: "not implemented", -8: "workspace null, misaligned or too small",
          -9: "page id, length or offset outside its range"}


class DsparkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed with status {code} ({STATUS.get(code, 'unknown')})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libdspark.so (building it first if asked); raises if unavailable."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing:
            path = _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libdspark.so not found at {path}; run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        P, i32, u64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float, ctypes.c_size_t
        L.dspark_strerror.argtypes = [i32]
        L.dspark_strerror.restype = ctypes.c_char_p
        L.dspark_version.restype = ctypes.c_char_p
        L.dspark_workspace_status.argtypes = [P, P]
        L.dspark_host_pointer.argtypes = [P, P]
        L.dspark_host_pointer.restype = i32
        L.dspark_draft_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.dspark_draft_workspace_size.restype = sz
        L.dspark_draft_markov.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, u64, P, f32,
                                          P, P, P, P, P, sz, P]
        L.dspark_draft_rnn.argtypes = [P, i32, P, P, P, P, i32, P, i32, i32, i32, i32, i32, u64, P, f32,
                                       P, P, P, P, P, P, sz, P]
        L.dspark_verify_workspace_size.argtypes = [i32, i32, i32, i32]
        L.dspark_verify_workspace_size.restype = sz
        L.dspark_verify.argtypes = [P, i32, P, i32, P, i32, P, P, P, P, P, i32, i32, i32, i32, u64, P, f32,
                                    P, P, P, P, P, P, sz, P]
        L.dspark_verify_staged.argtypes = [P, i32, P, i32, P, i32, P, P, P, P, P, i32, i32, i32, i32, u64, P, f32,
                                           P, P, P, P, P, P, P, sz, P]
        L.dspark_schedule_workspace_size.argtypes = [i32, i32]
        L.dspark_schedule_workspace_size.restype = sz
        L.dspark_draft_markov_conf.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, u64, P, f32,
                                               P, P, P, P, P, P, sz, P]
        L.dspark_draft_rnn_conf.argtypes = [P, i32, P, P, P, P, i32, P, i32, i32, i32, i32, i32, u64, P, f32,
                                            P, P, P, P, P, P, P, sz, P]
        L.dspark_schedule.argtypes = [P, P, i32, i32, i32, P, P, P, P, sz, P]
        L.dspark_schedule_async.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, sz, P]
        L.dspark_schedule_threshold.argtypes = [P, i32, i32, f32, i32, P, P]
        L.dspark_sts_workspace_size.argtypes = [i32, i32, i32, i32]
        L.dspark_sts_workspace_size.restype = sz
        L.dspark_sts_fit.argtypes = [P, P, i32, i32, P, i32, i32, P, P, P, P, P, sz, P]
        L.dspark_sts_apply.argtypes = [P, i32, i32, P, P, P]
        L.dspark_philox4x32_10.argtypes = [P, P, P, i32, P]
        i64 = ctypes.c_int64
        for name in ("dspark_kv_workspace_size", "dspark_attn_paged_workspace_size",
                     "dspark_attn_prompt_workspace_size"):
            getattr(L, name).argtypes = [] if name == "dspark_kv_workspace_size" else [i32] * 5
            getattr(L, name).restype = sz
        L.dspark_kv_write.argtypes = [P, P, P, P, i64, i64, P, sz, P]
        L.dspark_kv_read.argtypes = [P, P, P, P, P, sz, P]
        L.dspark_attn_paged.argtypes = [P, i64, P, P, i32, f32, P, P, P, sz, P]
        L.dspark_attn_prompt.argtypes = [P, P, P, i64, i64, i64, P, i32, i32, i32, i32, i32, f32, P, P, P, sz, P]
        L.dspark_attn_paged_window.argtypes = [P, i64, P, P, i32, f32, i32, i32, P, P, P, sz, P]
        L.dspark_attn_prompt_window.argtypes = [P, P, P, i64, i64, i64, P, i32, i32, i32, i32, i32, f32, i32, i32,
                                                P, P, P, sz, P]
        L.dspark_qk_rope.argtypes = [P, P, i64, i64, P, i32, i32, i32, i32, P, P, P, P, i64, i64, P]
        L.dspark_rope_write.argtypes = [P, P, P, P, P, i64, i64, i64, i32, P, P, P, P, P, i64, i64, P, sz, P]
        L.dspark_workspace_set_wait.argtypes = [P, u64, i32, P]
        L.dspark_profile_enable.argtypes = [i32]
        L.dspark_profile_collect.argtypes = [P, P, i32]
        L.dspark_profile_kernel_name.argtypes = [i32]
        L.dspark_profile_kernel_name.restype = ctypes.c_char_p
        for name in ("dspark_draft_markov", "dspark_draft_rnn", "dspark_draft_markov_conf", "dspark_draft_rnn_conf",
                     "dspark_verify", "dspark_verify_staged", "dspark_schedule", "dspark_schedule_async",
                     "dspark_schedule_threshold",
                     "dspark_sts_fit",
                     "dspark_sts_apply", "dspark_philox4x32_10", "dspark_workspace_set_wait",
                     "dspark_workspace_status", "dspark_profile_enable", "dspark_profile_collect",
                     "dspark_kv_write", "dspark_kv_read", "dspark_attn_paged", "dspark_attn_prompt",
                     "dspark_attn_paged_window", "dspark_attn_prompt_window", "dspark_qk_rope", "dspark_rope_write"):
            getattr(L, name).restype = i32
        _lib = L
        return _lib


class DeviceView:
    """A device-accessible address with a shape and a dtype, passed where the
    calls take a CUDA tensor: for example a pinned host buffer read in place
    (``host_view``)."""

    is_cuda = True

    def __init__(self, ptr: int, shape, dtype, device, owner=None):
        self.ptr, self.shape, self.dtype, self.device, self.owner = int(ptr), tuple(shape), dtype, device, owner

    def data_ptr(self) -> int:
        return self.ptr

    def is_contiguous(self) -> bool:
        return True

    def numel(self) -> int:
        n = 1
        for d in self.shape:
            n *= d
        return n


def host_view(t: torch.Tensor, device) -> DeviceView:
    """A pinned host tensor as a DeviceView its kernels read in place
    (``dspark_host_pointer``); raises if the memory is not pinned and mapped."""
    if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
        raise ValueError("host_view takes a contiguous pinned host tensor")
    out = ctypes.c_void_p()
    code = load().dspark_host_pointer(ctypes.c_void_p(t.data_ptr()), ctypes.byref(out))
    _check("dspark_host_pointer", code)
    return DeviceView(out.value, t.shape, t.dtype, device, owner=t)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdspark takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libdspark takes contiguous tensors")
    return t.data_ptr()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"storage dtype must be float32 or bfloat16, got {t.dtype}")


def _shape(name: str, t, shape, dtype=None):
    """The C ABI takes bare pointers and cannot see sizes: a tensor of the
    wrong shape would be read or written past its end on the device, so the
    binding checks every shape (and the dtype where it is fixed) first."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# The current stream's handle without a Stream object around it: 0.2 us on a
# GB300's host against 2.9 us, next to about 5 us for a call's own launches.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or _raw_device is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _check(fn: str, code: int):
    if code != 0:
        raise DsparkError(fn, code)


class _Conf(ctypes.Structure):
    """dspark_conf_t: the confidence head's arguments."""
    _fields_ = [("H", ctypes.c_void_p), ("w", ctypes.c_void_p), ("d", ctypes.c_int), ("c", ctypes.c_void_p),
                ("t", ctypes.c_void_p)]


def _conf(conf_w, conf_H, out, R, gamma, dev, conf_t=None, stream=None):
    """Fill out["c"] and return a dspark_conf_t pointer (None: head off)."""
    if conf_w is None:
        return None, None
    if conf_w.dtype != torch.float32:
        raise TypeError("confidence weights must be float32")
    if conf_H is not None and conf_H.dtype != torch.bfloat16:
        raise TypeError("confidence-head H must be bfloat16")
    if "c" not in out:
        out["c"] = _empty((R, gamma), torch.float32, dev, stream)
    if conf_t is not None and conf_t.dtype != torch.float64:
        raise TypeError("per-position temperatures must be float64")
    st = _Conf(_p(conf_H), _p(conf_w), 0 if conf_H is None else conf_H.shape[2], _p(out["c"]), _p(conf_t))
    return st, ctypes.byref(st)


def _on(stream, make):
    """What ``make()`` allocates and enqueues, on the stream of a call that was given
    one: on the current stream its zeros could come after the call's kernels, and
    its memory be that of earlier work which the call does not wait for.  The
    current stream, where the caller may use the result, is recorded."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _on(stream, lambda: torch.empty(shape, dtype=dtype, device=device))


def _workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    if stream is not None:
        return _on(stream, lambda: _workspace(nbytes, device))
    # torch's caching allocator returns 512-byte aligned blocks; the first
    # word (the device status word) must start at zero.
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def version() -> str:
    return load().dspark_version().decode()


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    return load().dspark_workspace_status(_p(ws), _stream(stream))


def workspace_set_wait(ws: torch.Tensor, limit_cycles: int = 0, test_withhold: int = 0, stream=None) -> None:
    """Bounded-wait limit (SM cycles, 0 = the default 2^32) and the test hook
    of the calls that use workspace ``ws`` (``dspark_workspace_set_wait``)."""
    code = load().dspark_workspace_set_wait(_p(ws), int(limit_cycles), int(test_withhold), _stream(stream))
    _check("dspark_workspace_set_wait", code)


def draft_workspace_bytes(R, gamma, V, r, d=0) -> int:
    return int(load().dspark_draft_workspace_size(R, gamma, V, r, d))


def verify_workspace_bytes(R, gamma, V, r) -> int:
    return int(load().dspark_verify_workspace_size(R, gamma, V, r))


def schedule_workspace_bytes(R, gamma) -> int:
    return int(load().dspark_schedule_workspace_size(R, gamma))


def _draft_shapes(R, gamma, V, r, anchor, W1, W2, req_ids):
    _shape("anchor", anchor, (R,), torch.int32)
    _shape("W1", W1, (V, r))
    _shape("W2", W2, (r, V))
    _shape("req_ids", req_ids, (R,))


def _draft_out_shapes(out, R, gamma, r):
    _shape("tokens", out["tokens"], (R, gamma), torch.int32)
    _shape("q_tok", out["q_tok"], (R, gamma), torch.float32)
    _shape("lse", out["lse"], (R, gamma), torch.float64)
    _shape("code", out["code"], (R, gamma, r), torch.float32)


def draft_markov(U, anchor, W1, W2, temperature: float, seed: int, req_ids=None, ws=None, out=None, stream=None,
                 conf_w=None, conf_H=None, conf_t=None):
    """Markov-head drafting (``dspark_draft_markov``).  Returns a dict of outputs.
    With ``conf_w`` ([d + r] float32) and ``conf_H`` ([R, gamma, d] bfloat16)
    the fused confidence head (``dspark_draft_markov_conf``) adds ``c``."""
    L = load()
    R, gamma, V = U.shape
    r = W1.shape[1]
    dev = U.device
    _draft_shapes(R, gamma, V, r, anchor, W1, W2, req_ids)
    if out is None:
        out = dict(tokens=_empty((R, gamma), torch.int32, dev, stream),
                   q_tok=_empty((R, gamma), torch.float32, dev, stream),
                   lse=_empty((R, gamma), torch.float64, dev, stream),
                   code=_empty((R, gamma, r), torch.float32, dev, stream))
    _draft_out_shapes(out, R, gamma, r)
    nbytes = L.dspark_draft_workspace_size(R, gamma, V, r, 0)
    if ws is None:
        ws = _workspace(nbytes, dev, stream)
    keep, cp = _conf(conf_w, conf_H, out, R, gamma, dev, conf_t, stream)
    code = L.dspark_draft_markov_conf(_p(U), _dt(U), _p(anchor), _p(W1), _p(W2), _dt(W1), R, gamma, V, r,
                                      int(seed) & 0xFFFFFFFFFFFFFFFF, _p(req_ids), float(temperature),
                                      _p(out["tokens"]), _p(out["q_tok"]), _p(out["lse"]), _p(out["code"]),
                                      cp, _p(ws), ws.numel(), _stream(stream))
    _check("dspark_draft_markov", code)
    out["ws"] = ws
    return out


def draft_rnn(U, anchor, W1, W2, Wgco, H, temperature: float, seed: int, req_ids=None, ws=None, out=None,
              stream=None, conf_w=None, conf_H=None, conf_t=None):
    """RNN-head drafting (``dspark_draft_rnn``).  With ``conf_w`` the fused
    confidence head adds ``c`` (``conf_H`` None: the head's own H)."""
    L = load()
    R, gamma, V = U.shape
    r = W1.shape[1]
    d = H.shape[2]
    dev = U.device
    if H.dtype != torch.bfloat16:
        raise TypeError("H must be bfloat16")
    _draft_shapes(R, gamma, V, r, anchor, W1, W2, req_ids)
    _shape("Wgco", Wgco, (2 * r + d, 3 * r))
    _shape("H", H, (R, gamma, d))
    if out is None:
        out = dict(tokens=_empty((R, gamma), torch.int32, dev, stream),
                   q_tok=_empty((R, gamma), torch.float32, dev, stream),
                   lse=_empty((R, gamma), torch.float64, dev, stream),
                   code=_empty((R, gamma, r), torch.float32, dev, stream),
                   state=_empty((R, r), torch.float32, dev, stream))
    _draft_out_shapes(out, R, gamma, r)
    _shape("state", out.get("state"), (R, r), torch.float32)
    nbytes = L.dspark_draft_workspace_size(R, gamma, V, r, d)
    if ws is None:
        ws = _workspace(nbytes, dev, stream)
    keep, cp = _conf(conf_w, conf_H, out, R, gamma, dev, conf_t, stream)
    code = L.dspark_draft_rnn_conf(_p(U), _dt(U), _p(anchor), _p(W1), _p(W2), _p(Wgco), _dt(W1), _p(H), d,
                                   R, gamma, V, r, int(seed) & 0xFFFFFFFFFFFFFFFF, _p(req_ids), float(temperature),
                                   _p(out["tokens"]), _p(out["q_tok"]), _p(out["lse"]), _p(out["code"]),
                                   _p(out.get("state")), cp, _p(ws), ws.numel(), _stream(stream))
    _check("dspark_draft_rnn", code)
    out["ws"] = ws
    return out


def verify(P, U, W2, draft, temperature: float, seed: int, verify_len=None, req_ids=None, ws=None, out=None,
           stream=None, p_stage=None):
    """Rejection-sampling verification (``dspark_verify``); ``draft`` is a draft output dict.
    ``p_stage`` (a device tensor of P's shape and dtype) receives the target
    rows pass 1 reads, for the later passes (``dspark_verify_staged``)."""
    L = load()
    R, G1, V = P.shape
    gamma = G1 - 1
    r = W2.shape[0]
    dev = P.device
    _shape("W2", W2, (r, V))
    if float(temperature) > 0.0:
        _shape("U", U, (R, gamma, V))
    _shape("draft tokens", draft["tokens"], (R, gamma), torch.int32)
    _shape("draft q_tok", draft.get("q_tok"), (R, gamma), torch.float32)
    _shape("draft lse", draft.get("lse"), (R, gamma), torch.float64)
    _shape("draft code", draft.get("code"), (R, gamma, r), torch.float32)
    _shape("verify_len", verify_len, (R,), torch.int32)
    _shape("req_ids", req_ids, (R,))
    if p_stage is not None:
        _shape("p_stage", p_stage, (R, G1, V), P.dtype)
    if out is None:
        out = dict(out_tokens=_empty((R, G1), torch.int32, dev, stream),
                   accept_len=_empty((R,), torch.int32, dev, stream),
                   n_out=_empty((R,), torch.int32, dev, stream),
                   p_tok=_empty((R, gamma), torch.float32, dev, stream),
                   lse_p=_empty((R, G1), torch.float64, dev, stream))
    _shape("out_tokens", out["out_tokens"], (R, G1), torch.int32)
    _shape("accept_len", out["accept_len"], (R,), torch.int32)
    _shape("n_out", out["n_out"], (R,), torch.int32)
    _shape("p_tok", out.get("p_tok"), (R, gamma), torch.float32)
    _shape("lse_p", out.get("lse_p"), (R, G1), torch.float64)
    nbytes = L.dspark_verify_workspace_size(R, gamma, V, r)
    if ws is None:
        ws = _workspace(nbytes, dev, stream)
    code = L.dspark_verify_staged(_p(P), _dt(P), _p(U), _dt(U), _p(W2), _dt(W2), _p(draft["tokens"]),
                                  _p(draft["q_tok"]), _p(draft["lse"]), _p(draft["code"]), _p(verify_len),
                                  R, gamma, V, r, int(seed) & 0xFFFFFFFFFFFFFFFF, _p(req_ids), float(temperature),
                                  _p(out["out_tokens"]), _p(out["accept_len"]), _p(out["n_out"]),
                                  _p(out.get("p_tok")), _p(out.get("lse_p")), _p(p_stage), _p(ws), ws.numel(),
                                  _stream(stream))
    _check("dspark_verify", code)
    out["ws"] = ws
    return out


def schedule(c, sps, ws=None, out=None, stream=None, budget=None):
    """Confidence scheduler (``dspark_schedule``): verify lengths, Theta*, n*.
    With ``budget`` (an int32 [1] device tensor: the n_star of two steps back)
    the production-style rule (``dspark_schedule_async``)."""
    L = load()
    R, gamma = c.shape
    dev = c.device
    if out is None:
        out = dict(verify_len=_empty((R,), torch.int32, dev, stream),
                   theta=_empty((1,), torch.float64, dev, stream),
                   n_star=_empty((1,), torch.int32, dev, stream))
    if ws is None:
        ws = _workspace(L.dspark_schedule_workspace_size(R, gamma), dev, stream)
    if budget is None:
        code = L.dspark_schedule(_p(c), _p(sps), sps.numel(), R, gamma, _p(out["verify_len"]), _p(out["theta"]),
                                 _p(out["n_star"]), _p(ws), ws.numel(), _stream(stream))
        _check("dspark_schedule", code)
    else:
        if budget.dtype != torch.int32:
            raise TypeError("budget must be int32")
        code = L.dspark_schedule_async(_p(c), _p(sps), sps.numel(), R, gamma, _p(budget), _p(out["verify_len"]),
                                       _p(out["theta"]), _p(out["n_star"]), _p(ws), ws.numel(), _stream(stream))
        _check("dspark_schedule_async", code)
    out["ws"] = ws
    return out


def schedule_threshold(c, theta: float, mode: int = 0, out=None, stream=None):
    """Threshold filter (``dspark_schedule_threshold``): per-request verify
    lengths, the longest prefix with a_{r,j} >= theta (mode 0) or
    c_{r,j} >= theta (mode 1)."""
    L = load()
    R, gamma = c.shape
    if out is None:
        out = _empty((R,), torch.int32, c.device, stream)
    code = L.dspark_schedule_threshold(_p(c), R, gamma, float(theta), int(mode), _p(out), _stream(stream))
    _check("dspark_schedule_threshold", code)
    return out


def sts_fit(c, accept_len, grid, M: int = 15, ws=None, out=None, stream=None):
    """Sequential Temperature Scaling (``dspark_sts_fit``): per-position
    temperatures t, grid indices g, minimum ECE and the gap to the second."""
    L = load()
    N, gamma = c.shape
    G = grid.numel()
    dev = c.device
    if grid.dtype != torch.float64 or accept_len.dtype != torch.int32:
        raise TypeError("grid must be float64 and accept_len int32")
    if out is None:
        out = dict(t=_empty((gamma,), torch.float64, dev, stream),
                   g=_empty((gamma,), torch.int32, dev, stream),
                   ece=_empty((gamma,), torch.float64, dev, stream),
                   gap=_empty((gamma,), torch.float64, dev, stream))
    if ws is None:
        ws = _workspace(L.dspark_sts_workspace_size(N, gamma, G, M), dev, stream)
    code = L.dspark_sts_fit(_p(c), _p(accept_len), N, gamma, _p(grid), G, M, _p(out["t"]), _p(out["g"]),
                            _p(out["ece"]), _p(out["gap"]), _p(ws), ws.numel(), _stream(stream))
    _check("dspark_sts_fit", code)
    out["ws"] = ws
    return out


def sts_apply(c, t, out=None, stream=None):
    """out = sigmoid(logit(c) / t[k]) per position (``dspark_sts_apply``)."""
    L = load()
    N, gamma = c.shape
    if out is None:
        out = _empty(c.shape, c.dtype, c.device, stream)
    code = L.dspark_sts_apply(_p(c), N, gamma, _p(t), _p(out), _stream(stream))
    _check("dspark_sts_apply", code)
    return out


class _Cache(ctypes.Structure):
    """dspark_kv_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("page", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class _Batch(ctypes.Structure):
    """dspark_kv_batch_t."""
    _fields_ = [("q_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("R", ctypes.c_int), ("max_pages", ctypes.c_int), ("T", ctypes.c_int)]


class KvCache:
    """One layer's paged key-value cache: k and v [n_pages, n_kv_heads, page,
    head_dim] in bfloat16 or float8_e4m3fn; the latter with float32 scales
    k_scale and v_scale [n_pages, n_kv_heads, page]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        f8 = k.dtype == torch.float8_e4m3fn
        if not f8 and k.dtype != torch.bfloat16:
            raise TypeError(f"the cache must be bfloat16 or float8_e4m3fn, got {k.dtype}")
        shape = k.shape
        if len(shape) != 4:
            raise ValueError("the cache must have shape (n_pages, n_kv_heads, page, head_dim)")
        _shape("v", v, shape, k.dtype)
        if f8 != (k_scale is not None):
            raise ValueError("k_scale goes with a float8_e4m3fn cache, and only with one")
        if f8 != (v_scale is not None):
            raise ValueError("v_scale goes with a float8_e4m3fn cache, and only with one")
        if f8:
            _shape("k_scale", k_scale, shape[:3], torch.float32)
            _shape("v_scale", v_scale, shape[:3], torch.float32)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page, self.head_dim = shape

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page: int, head_dim: int, dtype=torch.bfloat16, device="cuda"):
        """A new cache; its memory is not cleared (unwritten places are never read)."""
        shape = (n_pages, n_kv_heads, page, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        return cls(k, v, *(torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    def _struct(self) -> _Cache:
        return _Cache(_p(self.k), _p(self.v), _p(self.k_scale), _p(self.v_scale), BF16 if self.k_scale is None else E4M3,
                      self.n_pages, self.page, self.n_kv_heads, self.head_dim)


def _batch(q_off, kv_len, page_table, T) -> _Batch:
    if page_table.dim() != 2:
        raise ValueError("page_table must have shape (R, max_pages)")
    R, max_pages = page_table.shape
    if page_table.dtype != torch.int32:
        raise TypeError(f"page_table must be {torch.int32}, got {page_table.dtype}")
    _shape("q_off", q_off, (R + 1,), torch.int32)
    _shape("kv_len", kv_len, (R,), torch.int32)
    return _Batch(_p(q_off), _p(kv_len), _p(page_table), R, max_pages, T)


def _token_rows(name: str, t, T, heads, dim):
    """Data pointer and token stride of a bf16 [T, heads, dim] tensor whose
    tokens may be strided (a slice of a fused projection)."""
    _shape(name, t, (T, heads, dim), torch.bfloat16)
    if not t.is_cuda:
        raise ValueError("libdspark takes CUDA tensors")
    if T == 0:
        return t.data_ptr(), heads * dim
    step, head, one = t.stride()
    if one != 1 or (head != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (step if T > 1 else heads * dim)


def kv_write(cache: KvCache, K, V, q_off, kv_len, page_table, ws=None, stream=None):
    """Write new tokens' keys and values into the cache (``dspark_kv_write``);
    returns the workspace (its status word records bad pages)."""
    L = load()
    T = K.shape[0]
    b = _batch(q_off, kv_len, page_table, T)
    kp, ks = _token_rows("K", K, T, cache.n_kv_heads, cache.head_dim)
    vp, vs = _token_rows("V", V, T, cache.n_kv_heads, cache.head_dim)
    c = cache._struct()
    if ws is None:
        ws = _workspace(L.dspark_kv_workspace_size(), cache.k.device, stream)
    code = L.dspark_kv_write(ctypes.byref(c), ctypes.byref(b), kp, vp, ks, vs, _p(ws), ws.numel(), _stream(stream))
    _check("dspark_kv_write", code)
    return ws


def kv_read(cache: KvCache, kv_off, page_table, n_tokens: int, ws=None, out=None, stream=None):
    """Cached tokens back as bf16 (``dspark_kv_read``): request r's first
    kv_off[r+1] - kv_off[r] tokens go to rows kv_off[r].. of K and V
    [n_tokens, n_kv_heads, head_dim]."""
    L = load()
    shape = (n_tokens, cache.n_kv_heads, cache.head_dim)
    b = _batch(kv_off, None, page_table, n_tokens)
    if out is None:
        out = {name: _empty(shape, torch.bfloat16, cache.k.device, stream) for name in ("K", "V")}
    for name in ("K", "V"):
        _shape(name, out[name], shape, torch.bfloat16)
    c = cache._struct()
    if ws is None:
        ws = _workspace(L.dspark_kv_workspace_size(), cache.k.device, stream)
    code = L.dspark_kv_read(ctypes.byref(c), ctypes.byref(b), _p(out["K"]), _p(out["V"]), _p(ws), ws.numel(),
                            _stream(stream))
    _check("dspark_kv_read", code)
    out["ws"] = ws
    return out


def _attn_out(out, lse, T, heads, dim, dev, stream=None):
    if out is None:
        out = dict(out=_empty((T, heads, dim), torch.bfloat16, dev, stream))
        if lse:
            out["lse"] = _empty((T, heads), torch.float32, dev, stream)
        return out
    _shape("out", out["out"], (T, heads, dim), torch.bfloat16)
    _shape("lse", out.get("lse"), (T, heads), torch.float32)
    return out


def _window(window, sinks):
    """The extra arguments of a call with a window."""
    if window is None:
        if sinks:
            raise ValueError("sinks go with a window")
        return ()
    # longer than any request is as good as the longest the ABI can say, and what is below
    # its range is refused like the lowest in it
    return tuple(max(-1 << 31, min(int(n), 0x7FFFFFFF)) for n in (window, sinks))


def attn_paged(q, cache: KvCache, q_off, kv_len, page_table, scale: Optional[float] = None, lse: bool = False,
               ws=None, out=None, stream=None, window: Optional[int] = None, sinks: int = 0):
    """Attention of the new tokens q [T, n_heads, head_dim] over the paged
    cache (``dspark_attn_paged``); ``scale`` None: 1 / sqrt(head_dim).  With a
    ``window`` a token sees the last ``window`` tokens and the first ``sinks``
    alone (``dspark_attn_paged_window``).  Returns a dict with ``out`` and, on
    request, ``lse`` [T, n_heads]."""
    L = load()
    T, heads, dim = q.shape
    b = _batch(q_off, kv_len, page_table, T)
    qp, qs = _token_rows("q", q, T, heads, cache.head_dim)
    out = _attn_out(out, lse, T, heads, dim, q.device, stream)
    c = cache._struct()
    if ws is None:
        ws = _workspace(L.dspark_attn_paged_workspace_size(b.R, T, heads, cache.n_kv_heads, dim), q.device, stream)
    local = _window(window, sinks)
    name = "dspark_attn_paged_window" if local else "dspark_attn_paged"
    code = getattr(L, name)(qp, qs, ctypes.byref(c), ctypes.byref(b), heads, float(dim ** -0.5 if scale is None else scale),
                            *local, _p(out["out"]), _p(out.get("lse")), _p(ws), ws.numel(), _stream(stream))
    _check(name, code)
    out["ws"] = ws
    return out


def attn_prompt(q, k, v, seq_off, scale: Optional[float] = None, lse: bool = False, ws=None, out=None, stream=None,
                window: Optional[int] = None, sinks: int = 0):
    """Causal attention over whole packed prompts (``dspark_attn_prompt``, with a
    ``window`` ``dspark_attn_prompt_window``): q [T, n_heads, head_dim], k and v
    [T, n_kv_heads, head_dim], sequence b the tokens seq_off[b] ..
    seq_off[b+1].  Window and result as ``attn_paged``."""
    L = load()
    T, heads, dim = q.shape
    if k.dim() != 3:
        raise ValueError("k must have shape (T, n_kv_heads, head_dim)")
    kv_heads = k.shape[1]
    B = seq_off.numel() - 1
    _shape("seq_off", seq_off, (B + 1,), torch.int32)
    qp, qs = _token_rows("q", q, T, heads, dim)
    kp, ks = _token_rows("k", k, T, kv_heads, dim)
    vp, vs = _token_rows("v", v, T, kv_heads, dim)
    out = _attn_out(out, lse, T, heads, dim, q.device, stream)
    if ws is None:
        ws = _workspace(L.dspark_attn_prompt_workspace_size(B, T, heads, kv_heads, dim), q.device, stream)
    local = _window(window, sinks)
    name = "dspark_attn_prompt_window" if local else "dspark_attn_prompt"
    code = getattr(L, name)(qp, kp, vp, qs, ks, vs, _p(seq_off), B, T, heads, kv_heads, dim,
                            float(dim ** -0.5 if scale is None else scale), *local, _p(out["out"]), _p(out.get("lse")),
                            _p(ws), ws.numel(), _stream(stream))
    _check(name, code)
    out["ws"] = ws
    return out


class _Rope(ctypes.Structure):
    """dspark_rope_t."""
    _fields_ = [("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("axis", ctypes.c_uint8 * 64), ("inv_freq", ctypes.c_double * 64)]


class _HeadNorm(ctypes.Structure):
    """dspark_head_norm_t."""
    _fields_ = [("q_w", ctypes.c_void_p), ("k_w", ctypes.c_void_p), ("w_dtype", ctypes.c_int), ("eps", ctypes.c_float)]


class Rope:
    """Rotary positions: the first ``2 * len(inv_freq)`` values of a head are
    turned, pair i by position[axis[i]] * inv_freq[i] radians (``dspark_rope_t``).
    ``axis`` None: one axis.  ``interleaved`` pairs neighbours instead of the two
    halves; ``amplitude`` multiplies what is turned.  ``n_axes`` None: as many as
    ``axis`` names."""

    def __init__(self, inv_freq, axis=None, interleaved: bool = False, amplitude: float = 1.0,
                 n_axes: Optional[int] = None):
        inv_freq = [float(f) for f in inv_freq]
        axis = [0] * len(inv_freq) if axis is None else [int(a) for a in axis]
        if not 1 <= len(inv_freq) <= 64:
            raise ValueError(f"1 to 64 frequencies, got {len(inv_freq)}")
        if len(axis) != len(inv_freq) or min(axis) < 0 or max(axis) > 3:
            raise ValueError("axis must hold a number from 0 to 3 for each frequency")
        self._c = _Rope(2 * len(inv_freq), int(interleaved), max(axis) + 1 if n_axes is None else int(n_axes), amplitude,
                        (ctypes.c_uint8 * 64)(*axis), (ctypes.c_double * 64)(*inv_freq))
        self._ref = ctypes.byref(self._c)

    @property
    def n_axes(self) -> int:
        """Axes of the positions that it takes (fixed, like the rest of it)."""
        return self._c.n_axes

    @classmethod
    def from_theta(cls, rot: int, theta: float = 10000.0, **kw) -> "Rope":
        """The usual frequencies theta^(-2 i / rot), i < rot / 2."""
        return cls([theta ** (-2.0 * i / rot) for i in range(rot // 2)], **kw)


class HeadNorm:
    """RMS norm of each query and key head with weights ``q`` and ``k``
    [head_dim], float32 or bfloat16 CUDA tensors (None: that side is not normed).
    Each call takes the weights and ``eps`` as they are then: a module that was
    moved, cast or given other weights needs no new one."""

    def __init__(self, q=None, k=None, eps: float = 1e-6):
        self.q, self.k, self.eps = q, k, eps
        self._c = _HeadNorm()
        self._ref = ctypes.byref(self._c)
        self._arg()

    def _arg(self, dim: Optional[int] = None):
        """The struct, filled anew (a new one for each call takes a microsecond longer)."""
        q, k = self.q, self.k
        one = k if q is None else q
        if one is None:
            raise ValueError("HeadNorm takes weights for queries, keys or both")
        if (k is not None and k.dtype != one.dtype) or (dim is None and any(w is not None and w.dim() != 1 for w in (q, k))):
            raise ValueError("the weights must be vectors of one dtype")
        if dim is not None:
            _shape("the norm's q", q, (dim,))
            _shape("the norm's k", k, (dim,))
        c = self._c
        c.q_w, c.k_w, c.w_dtype, c.eps = _p(q), _p(k), _dt(one), self.eps
        return self._ref


def _turn_args(rope, norm, positions, T, dim):
    """Checks of what both calls share; the positions' and the structs' addresses."""
    if norm is not None:
        norm = norm._arg(dim)
    if positions is not None:
        if rope is None:
            raise ValueError("positions go with a rope")
        axes = rope.n_axes
        _shape("positions", positions, (T,) if axes == 1 and positions.dim() == 1 else (T, axes), torch.int32)
    return _p(positions), rope and rope._ref, norm


def _rows_out(out, name, T, heads, dim, dev, stream=None):
    """The output rows of that name, made if need be, with their address and stride."""
    if out.get(name) is None:
        t = out[name] = _empty((T, heads, dim), torch.bfloat16, dev, stream)
        return t.data_ptr(), heads * dim
    return _token_rows(name, out[name], T, heads, dim)


def qk_rope(q, k, positions, rope: Optional[Rope] = None, norm: Optional[HeadNorm] = None, out=None, stream=None):
    """Norm and rotation of query and key heads (``dspark_qk_rope``): q [T,
    n_heads, head_dim] and k [T, n_kv_heads, head_dim] (or None) in bf16,
    positions int32 [T] or [T, axes].  Returns a dict with ``q`` and ``k``;
    ``out=dict(q=q, k=k)`` works in place."""
    L = load()
    T, heads, dim = q.shape
    pos, rp, np_ = _turn_args(rope, norm, positions, T, dim)
    if rope is not None and positions is None:
        raise ValueError("a rope takes positions")
    out = {} if out is None else out
    qp, qs = _token_rows("q", q, T, heads, dim)
    qo, qos = _rows_out(out, "q", T, heads, dim, q.device, stream)
    kv_heads = kp = ks = ko = kos = 0
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k must have shape (T, n_kv_heads, head_dim)")
        kv_heads = k.shape[1]
        kp, ks = _token_rows("k", k, T, kv_heads, dim)
        ko, kos = _rows_out(out, "k", T, kv_heads, dim, q.device, stream)
    code = L.dspark_qk_rope(qp, kp or None, qs, ks, pos, T, heads, kv_heads, dim, rp, np_, qo, ko or None, qos, kos,
                            _stream(stream))
    _check("dspark_qk_rope", code)
    return out


def rope_write(cache: KvCache, q, K, V, q_off, kv_len, page_table, rope: Optional[Rope] = None,
               norm: Optional[HeadNorm] = None, positions=None, keep: bool = False, ws=None, out=None, stream=None):
    """Norm and rotation on the way into the cache (``dspark_rope_write``): K and V
    go to their pages as ``kv_write`` takes them, K normed and turned; q (None:
    keys and values alone) comes back in the dict's ``q``, with ``keep`` the turned
    keys in ``k``.  ``positions`` None: a token's place in its request; else
    [T] or [T, axes].  ``ws`` holds the status word, as for ``kv_write``."""
    L = load()
    T, dim = K.shape[0], cache.head_dim
    b = _batch(q_off, kv_len, page_table, T)
    pos, rp, np_ = _turn_args(rope, norm, positions, T, dim)
    out = {} if out is None else out
    dev = cache.k.device
    kp, ks = _token_rows("K", K, T, cache.n_kv_heads, dim)
    vp, vs = _token_rows("V", V, T, cache.n_kv_heads, dim)
    heads = qs = qos = kos = 0
    qp = qo = ko = None
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must have shape (T, n_heads, head_dim)")
        heads = q.shape[1]
        qp, qs = _token_rows("q", q, T, heads, dim)
        qo, qos = _rows_out(out, "q", T, heads, dim, dev, stream)
    if keep or out.get("k") is not None:
        ko, kos = _rows_out(out, "k", T, cache.n_kv_heads, dim, dev, stream)
    c = cache._struct()
    if ws is None:
        ws = _workspace(L.dspark_kv_workspace_size(), dev, stream)
    code = L.dspark_rope_write(ctypes.byref(c), ctypes.byref(b), qp, kp, vp, qs, ks, vs, heads, pos, rp, np_, qo, ko, qos, kos,
                               _p(ws), ws.numel(), _stream(stream))
    _check("dspark_rope_write", code)
    out["ws"] = ws
    return out


def philox4x32_10(ctr, key, out=None, stream=None):
    """The device's Philox4x32-10 block function on n counters ``ctr`` [n, 4]
    and keys ``key`` [n, 2] (uint32 values in int32 CUDA tensors, bit for
    bit); returns out [n, 4] (``dspark_philox4x32_10``)."""
    L = load()
    n = ctr.shape[0]
    _shape("ctr", ctr, (n, 4), torch.int32)
    _shape("key", key, (n, 2), torch.int32)
    if out is None:
        out = _empty((n, 4), torch.int32, ctr.device, stream)
    _shape("out", out, (n, 4), torch.int32)
    code = L.dspark_philox4x32_10(_p(ctr), _p(key), _p(out), n, _stream(stream))
    _check("dspark_philox4x32_10", code)
    return out


def profile_enable(on: bool = True) -> None:
    """Bracket every library launch with CUDA events (benchmark timing)."""
    load().dspark_profile_enable(1 if on else 0)


def profile_collect(cap: int = 1 << 16):
    """Per launch since the last collect: list of (kernel name, milliseconds)."""
    import numpy as np
    L = load()
    ids = np.zeros(cap, np.int32)
    ms = np.zeros(cap, np.float32)
    n = L.dspark_profile_collect(ctypes.c_void_p(ids.ctypes.data), ctypes.c_void_p(ms.ctypes.data), cap)
    if n < 0:
        raise DsparkError("dspark_profile_collect", n)
    n = min(n, cap)
    return [(L.dspark_profile_kernel_name(int(i)).decode(), float(t)) for i, t in zip(ids[:n], ms[:n])]
