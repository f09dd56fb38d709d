"""GB300 (sm_103a) large-chunk TTT-KVB layer and chunked linear attention.

Thin ctypes binding over the C ABI in ``include/``: every step of the
computation runs in the library's CUDA kernels; this module only marshals
arguments (device pointers of torch tensors, the current CUDA stream) and
allocates outputs and workspace with torch.  There is no CPU fallback: if the
shared library is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Sequence

import torch

APPLY_THEN_UPDATE = 0
BLOCK_CAUSAL = 1
BIDIRECTIONAL = 2
STRIDED = 3

TTT_F32 = 0
TTT_BF16 = 1

MUON_COEF = (3.4445, -4.7750, 2.0315)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libttt_gb300.so")

# Every symbol the public headers declare.
EXPORTED = (
    "ttt_status_string", "ttt_layer_workspace_size", "ttt_layer_forward",
    "linattn_workspace_size", "linattn_chunked_forward", "ttt_device_status",
    "ttt_set_wait_limit_ns", "ttt_selftest_gemm", "ttt_launch_count", "ttt_profile_start",
    "ttt_profile_stop", "linattn_chunked_forward_noalloc", "ttt_layer_host_workspace_size",
    "ttt_layer_forward_host", "ttt_selftest_withhold_release", "linattn_rule_workspace_size",
    "linattn_chunked_forward_rule", "delta_rule_workspace_size", "delta_rule_chunked_forward",
    "delta_rule_step", "block_norm_forward", "ttt_selftest_withhold_delta",
    "window_attention_forward", "window_attention_step", "selective_scan_workspace_size",
    "selective_scan_forward", "selective_scan_step", "short_conv_forward", "short_conv_step",
    "ttt_selftest_withhold_window",
)


class ProfileEntry(ctypes.Structure):
    """Mirror of ``ttt_profile_entry``."""
    _fields_ = [("name", ctypes.c_char * 32), ("kernel", ctypes.c_char * 32),
                ("launches", ctypes.c_int), ("ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double),
                ("sm_ms", ctypes.c_double)]


FORM_AUTO = 0
FORM_RECURRENT = 1
FORM_PARALLEL = 2


GATE_NONE = 0
GATE_SILU = 1
GATE_SIGMOID = 2


class UpdateRule(ctypes.Structure):
    """Mirror of ``ttt_update_rule``."""
    _fields_ = [("l2norm", ctypes.c_int), ("muon_steps", ctypes.c_int),
                ("momentum_beta", ctypes.c_float), ("ns_a", ctypes.c_float),
                ("ns_b", ctypes.c_float), ("ns_c", ctypes.c_float),
                ("last_layer_only", ctypes.c_int), ("inner_steps", ctypes.c_int),
                ("form", ctypes.c_int)]


class LinattnRule(ctypes.Structure):
    """Mirror of ``linattn_rule``."""
    _fields_ = [("alpha", ctypes.c_void_p), ("lr", ctypes.c_void_p), ("M0", ctypes.c_void_p),
                ("M_final", ctypes.c_void_p), ("muon_steps", ctypes.c_int),
                ("ns_a", ctypes.c_float), ("ns_b", ctypes.c_float), ("ns_c", ctypes.c_float)]


def update_rule(l2norm=True, muon_steps=0, momentum_beta=0.0, ns_coef=MUON_COEF,
                last_layer_only=False, inner_steps=1, form=FORM_AUTO) -> UpdateRule:
    a, b, c = ns_coef
    return UpdateRule(int(bool(l2norm)), int(muon_steps), float(momentum_beta),
                      float(a), float(b), float(c), int(bool(last_layer_only)),
                      int(inner_steps), int(form))


class TTTError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} (status {code})")
        self.code = code


_lib = None


def _declare(lib):
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.ttt_status_string.restype = ctypes.c_char_p
    lib.ttt_status_string.argtypes = [i]
    lib.ttt_layer_workspace_size.restype = sz
    lib.ttt_layer_workspace_size.argtypes = [i, i, i, i, i, i, i, i, ctypes.POINTER(UpdateRule)]
    lib.ttt_layer_forward.restype = i
    lib.ttt_layer_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i,
                                      vp, ctypes.POINTER(UpdateRule), vp, vp, vp, vp, vp, vp,
                                      sz, vp]
    lib.ttt_layer_host_workspace_size.restype = sz
    lib.ttt_layer_host_workspace_size.argtypes = [i, i, i, i, i, i, i, i,
                                                  ctypes.POINTER(UpdateRule), i]
    lib.ttt_layer_forward_host.restype = i
    lib.ttt_layer_forward_host.argtypes = lib.ttt_layer_forward.argtypes
    lib.linattn_workspace_size.restype = sz
    lib.linattn_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.linattn_chunked_forward.restype = i
    lib.linattn_chunked_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp,
                                            vp, vp, vp, sz, vp]
    lib.linattn_rule_workspace_size.restype = sz
    lib.linattn_rule_workspace_size.argtypes = [i, i, i, i, i, i, i, i,
                                                ctypes.POINTER(LinattnRule)]
    lib.linattn_chunked_forward_rule.restype = i
    lib.linattn_chunked_forward_rule.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp,
                                                 ctypes.POINTER(LinattnRule), vp, vp, vp, sz, vp]
    lib.ttt_device_status.restype = i
    lib.ttt_device_status.argtypes = [vp]
    lib.ttt_set_wait_limit_ns.restype = None
    lib.ttt_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.ttt_selftest_gemm.restype = i
    lib.ttt_selftest_gemm.argtypes = [vp, vp, vp, i, i, i, i, i, i, i, i, vp]
    lib.linattn_chunked_forward_noalloc.restype = i
    lib.linattn_chunked_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i,
                                                    vp, vp, vp, vp]
    f32, ll = ctypes.c_float, ctypes.c_longlong   # strides: packed bytes (c_char_p)
    lib.delta_rule_workspace_size.restype = sz
    lib.delta_rule_workspace_size.argtypes = [i] * 8
    lib.delta_rule_chunked_forward.restype = i
    lib.delta_rule_chunked_forward.argtypes = [vp] * 7 + [i] * 8 + [
        f32, ctypes.c_char_p, vp, vp, vp, sz, vp]
    lib.delta_rule_step.restype = i
    lib.delta_rule_step.argtypes = [vp] * 7 + [i] * 7 + [
        f32, ctypes.c_char_p, vp, vp]
    lib.block_norm_forward.restype = i
    lib.block_norm_forward.argtypes = [vp] * 6 + [ll] + [i] * 5 + [
        f32, ctypes.c_char_p, vp, vp, vp]
    cp = ctypes.c_char_p
    lib.window_attention_forward.restype = i
    lib.window_attention_forward.argtypes = [vp] * 6 + [i, vp, vp] + [i] * 9 + [f32, cp, vp, vp]
    lib.window_attention_step.restype = i
    lib.window_attention_step.argtypes = [vp] * 7 + [i] * 8 + [f32, cp, vp, vp]
    lib.selective_scan_workspace_size.restype = sz
    lib.selective_scan_workspace_size.argtypes = [i] * 7
    lib.selective_scan_forward.restype = i
    lib.selective_scan_forward.argtypes = [vp] * 10 + [i] * 8 + [cp, vp, vp, vp, sz, vp]
    lib.selective_scan_step.restype = i
    lib.selective_scan_step.argtypes = [vp] * 10 + [i] * 7 + [cp, vp, vp]
    lib.short_conv_forward.restype = i
    lib.short_conv_forward.argtypes = [vp] * 5 + [i] * 7 + [cp, vp, vp, vp]
    lib.short_conv_step.restype = i
    lib.short_conv_step.argtypes = [vp] * 5 + [i] * 6 + [cp, vp, vp]
    for name in ("window_forward", "window_step", "scan_forward", "scan_step", "conv_forward",
                 "conv_step"):   # the same calls with their arguments as one packed record
        call = getattr(lib, "ttt_binding_" + name)
        call.restype, call.argtypes = i, [cp]
    lib.ttt_binding_record_bytes.restype, lib.ttt_binding_record_bytes.argtypes = sz, [i]
    for which, record in enumerate(_RECORDS):
        if lib.ttt_binding_record_bytes(which) != record.size:
            raise RuntimeError(f"{LIB_PATH} does not belong to this binding: build it again")
    lib.ttt_selftest_withhold_delta.restype = None
    lib.ttt_selftest_withhold_delta.argtypes = [i]
    lib.ttt_selftest_withhold_window.restype = None
    lib.ttt_selftest_withhold_window.argtypes = [i]
    lib.ttt_selftest_withhold_release.restype = None
    lib.ttt_selftest_withhold_release.argtypes = [i]
    lib.ttt_launch_count.restype = ctypes.c_ulonglong
    lib.ttt_launch_count.argtypes = []
    lib.ttt_profile_start.restype = None
    lib.ttt_profile_start.argtypes = []
    lib.ttt_profile_stop.restype = i
    lib.ttt_profile_stop.argtypes = [ctypes.POINTER(ProfileEntry), i]
    return lib


def library():
    """Loads the shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library not built: {LIB_PATH} is missing "
                "(run chunked_linear_attention_gb300._build.build())")
        _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(code: int) -> str:
    return library().ttt_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the CUDA path must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _io_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TTT_BF16
    if t.dtype == torch.float32:
        return TTT_F32
    raise ValueError(f"unsupported I/O dtype {t.dtype}")


def _flags(update_chunks, n_chunks):
    if update_chunks is None:
        return None, None
    if len(update_chunks) != n_chunks:
        raise ValueError(f"update_chunks needs {n_chunks} flags, got {len(update_chunks)}")
    arr = (ctypes.c_ubyte * n_chunks)(*[1 if x else 0 for x in update_chunks])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def _check(rc: int, what: str):
    if rc != 0:
        raise TTTError(rc, what)


def layer_workspace_size(B, H, N, d_h, m_h, chunk, io_dtype, mask_mode, rule: UpdateRule) -> int:
    return library().ttt_layer_workspace_size(B, H, N, d_h, m_h, chunk, io_dtype, mask_mode,
                                              ctypes.byref(rule))


def ttt_layer_forward(q, k, v, eta, W1, W2, W3, chunk: int, mask_mode: int,
                      rule: Optional[UpdateRule] = None,
                      update_chunks: Optional[Sequence[int]] = None,
                      momentum: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None,
                      W_final: Optional[Sequence[torch.Tensor]] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """LaCT TTT layer forward (see ``ttt_layer_forward`` in include/ttt.h).

    q, k, v: [B, H, N, d] CUDA tensors (bf16 or fp32); eta [B, H, N] fp32;
    W1, W3 [H, m, d] or [B, H, m, d]; W2 [H, d, m] or [B, H, d, m], fp32.
    Returns (out, W1_final, W2_final, W3_final).  Asynchronous on the current
    stream (or ``stream``).
    """
    lib = library()
    rule = update_rule() if rule is None else rule
    B, H, N, d = q.shape
    m = W1.shape[-2]
    io = _io_dtype(q)
    w_per_batch = 1 if W1.dim() == 4 else 0
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if W_final is None:
        W_final = (torch.empty((B, H, m, d), device=dev, dtype=torch.float32),
                   torch.empty((B, H, d, m), device=dev, dtype=torch.float32),
                   torch.empty((B, H, m, d), device=dev, dtype=torch.float32))
    ws_bytes = lib.ttt_layer_workspace_size(B, H, N, d, m, chunk, io, mask_mode, ctypes.byref(rule))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    keep, fl = _flags(update_chunks, N // chunk if chunk > 0 else 0)
    rc = lib.ttt_layer_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(W1), _ptr(W2), _ptr(W3),
                               w_per_batch, B, H, N, d, m, chunk, io, mask_mode, fl,
                               ctypes.byref(rule), _ptr(out), _ptr(W_final[0]), _ptr(W_final[1]),
                               _ptr(W_final[2]), _ptr(momentum), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), _stream(stream))
    del keep
    _check(rc, "ttt_layer_forward")
    return out, W_final[0], W_final[1], W_final[2]


def _hptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("tensors passed to the host-buffer call must be in host memory")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if not t.is_pinned():
        raise ValueError("host tensors must be page-locked (tensor.pin_memory())")
    return ctypes.c_void_p(t.data_ptr())


def layer_host_workspace_size(B, H, N, d_h, m_h, chunk, io_dtype, mask_mode, rule: UpdateRule,
                              w_per_batch: int = 0) -> int:
    return library().ttt_layer_host_workspace_size(B, H, N, d_h, m_h, chunk, io_dtype, mask_mode,
                                                   ctypes.byref(rule), int(w_per_batch))


def ttt_layer_forward_host(q, k, v, eta, W1, W2, W3, chunk: int, mask_mode: int,
                           rule: Optional[UpdateRule] = None,
                           update_chunks: Optional[Sequence[int]] = None,
                           momentum: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None,
                           W_final: Optional[Sequence[torch.Tensor]] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None, device=None):
    """LaCT TTT layer forward on page-locked HOST tensors (see
    ``ttt_layer_forward_host`` in include/ttt.h): the same shapes as
    ``ttt_layer_forward``; chunk transfers overlap the kernels.  ``workspace``
    (a CUDA uint8 tensor) and ``stream`` select the device (else ``device`` or
    the current one).  Returns (out, W1_final, W2_final, W3_final) host
    tensors, complete once ``stream`` reaches this point.
    """
    lib = library()
    rule = update_rule() if rule is None else rule
    B, H, N, d = q.shape
    m = W1.shape[-2]
    io = _io_dtype(q)
    w_per_batch = 1 if W1.dim() == 4 else 0
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if W_final is None:
        W_final = (torch.empty((B, H, m, d), dtype=torch.float32, pin_memory=True),
                   torch.empty((B, H, d, m), dtype=torch.float32, pin_memory=True),
                   torch.empty((B, H, m, d), dtype=torch.float32, pin_memory=True))
    dev = workspace.device if workspace is not None else torch.device(
        "cuda", torch.cuda.current_device() if device is None else torch.device(device).index)
    ws_bytes = lib.ttt_layer_host_workspace_size(B, H, N, d, m, chunk, io, mask_mode,
                                                 ctypes.byref(rule), w_per_batch)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    keep, fl = _flags(update_chunks, N // chunk if chunk > 0 else 0)
    with torch.cuda.device(dev):
        rc = lib.ttt_layer_forward_host(
            _hptr(q), _hptr(k), _hptr(v), _hptr(eta), _hptr(W1), _hptr(W2), _hptr(W3),
            w_per_batch, B, H, N, d, m, chunk, io, mask_mode, fl, ctypes.byref(rule), _hptr(out),
            _hptr(W_final[0]), _hptr(W_final[1]), _hptr(W_final[2]), _hptr(momentum),
            _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))
    del keep
    _check(rc, "ttt_layer_forward_host")
    return out, W_final[0], W_final[1], W_final[2]


def linattn_workspace_size(B, H, N, d_k, d_v, chunk, io_dtype, mask_mode) -> int:
    return library().linattn_workspace_size(B, H, N, d_k, d_v, chunk, io_dtype, mask_mode)


def linattn_chunked_forward(q, k, v, eta, chunk: int, mask_mode: int,
                            S0: Optional[torch.Tensor] = None,
                            update_chunks: Optional[Sequence[int]] = None,
                            out: Optional[torch.Tensor] = None,
                            S_final: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None):
    """Chunked linear attention (see ``linattn_chunked_forward`` in include/ttt.h).

    Returns (out [B, H, N, d_v], S_final [B, H, d_v, d_k] fp32).
    """
    lib = library()
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    io = _io_dtype(q)
    dev = q.device
    if out is None:
        out = torch.empty((B, H, N, dv), device=dev, dtype=q.dtype)
    if S_final is None:
        S_final = torch.empty((B, H, dv, dk), device=dev, dtype=torch.float32)
    ws_bytes = lib.linattn_workspace_size(B, H, N, dk, dv, chunk, io, mask_mode)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    keep, fl = _flags(update_chunks, N // chunk if chunk > 0 else 0)
    rc = lib.linattn_chunked_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(S0), B, H, N, dk,
                                     dv, chunk, io, mask_mode, fl, _ptr(out), _ptr(S_final),
                                     _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                     _stream(stream))
    del keep
    _check(rc, "linattn_chunked_forward")
    return out, S_final


def linattn_rule(alpha=None, lr=None, M0=None, M_final=None, muon_steps=0,
                 ns_coef=MUON_COEF) -> LinattnRule:
    """The ``linattn_rule`` struct from CUDA tensors (or None)."""
    a, b, c = ns_coef
    return LinattnRule(_ptr(alpha), _ptr(lr), _ptr(M0), _ptr(M_final), int(muon_steps),
                       float(a), float(b), float(c))


def linattn_chunked_forward_rule(q, k, v, eta, chunk: int, mask_mode: int,
                                 S0: Optional[torch.Tensor] = None,
                                 update_chunks: Optional[Sequence[int]] = None,
                                 alpha: Optional[torch.Tensor] = None,
                                 lr: Optional[torch.Tensor] = None,
                                 M0: Optional[torch.Tensor] = None,
                                 M_final=None, muon_steps: int = 0, ns_coef=MUON_COEF,
                                 out: Optional[torch.Tensor] = None,
                                 S_final: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Chunked linear attention with momentum, per-chunk learning rates and
    Muon of the momentum (see ``linattn_chunked_forward_rule`` in
    include/ttt.h).  alpha, lr: [B, H, N / chunk] fp32 CUDA tensors or None;
    M0 [B, H, d_v, d_k] or None; M_final: a tensor to write, True to allocate
    one, or None.  Returns (out, S_final, M_final or None)."""
    lib = library()
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    io = _io_dtype(q)
    dev = q.device
    if out is None:
        out = torch.empty((B, H, N, dv), device=dev, dtype=q.dtype)
    if S_final is None:
        S_final = torch.empty((B, H, dv, dk), device=dev, dtype=torch.float32)
    if M_final is True:
        M_final = torch.empty((B, H, dv, dk), device=dev, dtype=torch.float32)
    rule = linattn_rule(alpha, lr, M0, M_final, muon_steps, ns_coef)
    ws_bytes = lib.linattn_rule_workspace_size(B, H, N, dk, dv, chunk, io, mask_mode,
                                               ctypes.byref(rule))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    keep, fl = _flags(update_chunks, N // chunk if chunk > 0 else 0)
    rc = lib.linattn_chunked_forward_rule(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(S0), B, H,
                                          N, dk, dv, chunk, io, mask_mode, fl, ctypes.byref(rule),
                                          _ptr(out), _ptr(S_final), _ptr(workspace),
                                          0 if workspace is None else workspace.numel(),
                                          _stream(stream))
    del keep
    _check(rc, "linattn_chunked_forward_rule")
    return out, S_final, M_final


def linattn_chunked_forward_noalloc(q, k, v, eta, chunk: int, mask_mode: int,
                                    S0: Optional[torch.Tensor] = None,
                                    update_chunks: Optional[Sequence[int]] = None,
                                    out: Optional[torch.Tensor] = None,
                                    S_final: Optional[torch.Tensor] = None, stream=None):
    """Chunked linear attention whose scratch is the library's fixed 16 MiB
    device array instead of a workspace (see
    ``linattn_chunked_forward_noalloc`` in include/ttt.h).  Output tensors are
    still the caller's (allocated here with torch when not given)."""
    lib = library()
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if out is None:
        out = torch.empty((B, H, N, dv), device=dev, dtype=q.dtype)
    if S_final is None:
        S_final = torch.empty((B, H, dv, dk), device=dev, dtype=torch.float32)
    keep, fl = _flags(update_chunks, N // chunk if chunk > 0 else 0)
    # the library looks up its scratch array on the CURRENT device: make it
    # the tensors' device for the call
    with torch.cuda.device(dev):
        rc = lib.linattn_chunked_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(eta), _ptr(S0),
                                                 B, H, N, dk, dv, chunk, _io_dtype(q), mask_mode,
                                                 fl, _ptr(out), _ptr(S_final),
                                                 _stream(stream))
    del keep
    _check(rc, "linattn_chunked_forward_noalloc")
    return out, S_final


# The delta-rule and norm calls are made once per layer and decoded token, so
# their bindings keep the host's share short: strides travel as packed bytes,
# and the stream is looked up by device index (None in a torch without CUDA, which
# has no tensors that get so far).
_pack_layout = struct.Struct("18q").pack
_pack_norm_strides = struct.Struct("5q").pack
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_BF16, _F32 = torch.bfloat16, torch.float32


def _elsewhere(dev, stream):
    """A context that makes `dev` current and `stream` too where one is given
    (outputs and workspace then belong to the stream that uses them)."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream must be on {dev}")
        return torch.cuda.stream(stream)
    return torch.cuda.device(dev)


def _want(t, shape, dtype, dev, what):
    if t.shape == shape and t.dtype is dtype and t.device == dev:
        return
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{what} must be on {dev}, got {t.device}")


def _dense(t, shape, dtype, dev, what):
    """Address of a contiguous tensor of this shape, or None for None."""
    if t is None:
        return None
    _want(t, shape, dtype, dev, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _strides(t, what):
    """Strides of a tensor whose last dimension is contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return st


def delta_rule_workspace_size(B, Hk, Hv, N, d_k, d_v, n_seq, io_dtype) -> int:
    return library().delta_rule_workspace_size(B, Hk, Hv, N, d_k, d_v, n_seq, io_dtype)


def delta_rule_chunked_forward(q, k, v, g, beta, S0: Optional[torch.Tensor] = None,
                               seq_starts: Optional[torch.Tensor] = None,
                               scale: Optional[float] = None,
                               out: Optional[torch.Tensor] = None,
                               S_final: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None):
    """The gated delta rule over whole sequences (see
    ``delta_rule_chunked_forward`` in include/ttt_delta.h).

    q, k [B, Hk, N, d_k] and v [B, Hv, N, d_v], bf16 or fp32, any strides with
    the last dimension contiguous; g (log decay), beta [B, Hv, N] fp32.
    seq_starts: int32 [n_seq + 1] on the same device for sequences packed
    along the token axis (B = 1).  scale: d_k ** -0.5 when None.  S0 and
    S_final [n_seq or B, Hv, d_v, d_k] fp32.  Without ``out``, the outputs are
    stored in v's order of dimensions.  Returns (out [B, Hv, N, d_v], S_final).
    """
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors passed to the CUDA path must be on a CUDA device")
    if stream is not None or dev.index != _current_device():
        with _elsewhere(dev, stream):
            return delta_rule_chunked_forward(q, k, v, g, beta, S0, seq_starts, scale, out,
                                              S_final, workspace)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must have four dimensions")
    B, Hk, N, dk = q.shape
    Hv, dv = v.shape[1], v.shape[3]
    dt, io, f32 = q.dtype, _io_dtype(q), _F32
    _want(k, (B, Hk, N, dk), dt, dev, "k")
    _want(v, (B, Hv, N, dv), dt, dev, "v")
    _want(g, (B, Hv, N), f32, dev, "g")
    _want(beta, (B, Hv, N), f32, dev, "beta")
    n_seq = B
    if seq_starts is not None:
        if B != 1:
            raise ValueError("seq_starts needs B = 1")
        n_seq = seq_starts.numel() - 1
        if n_seq < 1 or not seq_starts.is_contiguous():
            raise ValueError("seq_starts must be a contiguous vector of n_seq + 1 entries")
        _want(seq_starts, (n_seq + 1,), torch.int32, dev, "seq_starts")
    lib = _lib or library()
    if out is None:
        out = torch.empty_like(v)   # v's strides where they are dense, else row-major
    else:
        _want(out, (B, Hv, N, dv), dt, dev, "out")
    state = (n_seq, Hv, dv, dk)
    if S_final is None:
        S_final = torch.empty(state, device=dev, dtype=f32)
    if workspace is None:
        need = lib.delta_rule_workspace_size(B, Hk, Hv, N, dk, dv, n_seq, io)
        workspace = torch.empty(need or 256, device=dev, dtype=torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    rc = lib.delta_rule_chunked_forward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        _dense(S0, state, f32, dev, "S0"),
        None if seq_starts is None else seq_starts.data_ptr(), n_seq, B, Hk, Hv, N, dk, dv, io,
        dk ** -0.5 if scale is None else scale,
        _pack_layout(*_strides(q, "q")[:3], *_strides(k, "k")[:3], *_strides(v, "v")[:3],
                     *g.stride(), *beta.stride(), *_strides(out, "out")[:3]),
        out.data_ptr(), _dense(S_final, state, f32, dev, "S_final"), workspace.data_ptr(),
        workspace.nbytes,
        _raw_stream(dev.index))
    if rc:
        _check(rc, "delta_rule_chunked_forward")
    return out, S_final


def delta_rule_step(q, k, v, g, beta, state, slots: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    stream=None):
    """The gated delta rule for one token of each of B sequences, on a pool of
    states that is updated in place (see ``delta_rule_step`` in
    include/ttt_delta.h).

    q, k [B, Hk, d_k], v [B, Hv, d_v], bf16 or fp32, last dimension
    contiguous; g, beta [B, Hv] fp32; state [n_slots, Hv, d_v, d_k] fp32;
    slots int32 [B] (negative: an idle row) or None.  Returns out [B, Hv, d_v].
    """
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors passed to the CUDA path must be on a CUDA device")
    if stream is not None or dev.index != _current_device():
        with _elsewhere(dev, stream):
            return delta_rule_step(q, k, v, g, beta, state, slots, scale, out)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q and v must have three dimensions, state four")
    B, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    dt, io, f32 = q.dtype, _io_dtype(q), _F32
    _want(k, (B, Hk, dk), dt, dev, "k")
    _want(v, (B, Hv, dv), dt, dev, "v")
    _want(g, (B, Hv), f32, dev, "g")
    _want(beta, (B, Hv), f32, dev, "beta")
    n_slots = state.shape[0]
    if out is None:
        out = torch.empty_like(v)   # half the host time of torch.empty with a device
    else:
        _want(out, (B, Hv, dv), dt, dev, "out")
    rc = (_lib or library()).delta_rule_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        _dense(state, (n_slots, Hv, dv, dk), f32, dev, "state"),
        _dense(slots, (B,), torch.int32, dev, "slots"), n_slots, B, Hk, Hv, dk, dv, io,
        dk ** -0.5 if scale is None else scale,
        _pack_layout(*_strides(q, "q")[:2], 0, *_strides(k, "k")[:2], 0, *_strides(v, "v")[:2], 0,
                     *g.stride(), 0, *beta.stride(), 0, *_strides(out, "out")[:2], 0),
        out.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "delta_rule_step")
    return out


def _rows(t, rows, D, dtype, dev, what):
    """Row stride of a [..., D] tensor whose leading dimensions run on as one."""
    if t.dtype != dtype or t.device != dev:
        raise ValueError(f"{what} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
    if t.shape[-1] != D or t.numel() != rows * D:
        raise ValueError(f"{what} must hold {rows} rows of {D}, got shape {tuple(t.shape)}")
    if t.is_contiguous():
        return D
    strides = _strides(t, what)
    stride, size = None, 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * size:
            raise ValueError(f"the rows of {what} must be equally far apart")
        size *= n
    return D if stride is None else stride


def block_norm_forward(y, w: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, gate_act: int = GATE_NONE,
                       residual: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None,
                       w_next: Optional[torch.Tensor] = None, group: Optional[int] = None,
                       eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None,
                       out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                       stream=None):
    """The norms around a block with its gate, residual scale and residual sum
    (see ``block_norm_forward`` in include/ttt_delta.h).

    y, gate [..., D] bf16 or fp32; residual [..., D] and out in ``out_dtype``
    (residual's type, or y's); w [group] (its length sets the group), scale
    and w_next [D] fp32.  Returns (out, h); h is None without ``w_next``.
    """
    dev = y.device
    if dev.type != "cuda":
        raise ValueError("tensors passed to the CUDA path must be on a CUDA device")
    if stream is not None or dev.index != _current_device():
        with _elsewhere(dev, stream):
            return block_norm_forward(y, w, gate, gate_act, residual, scale, w_next, group, eps,
                                      out_dtype, out, h)
    D, n, dt, io, f32 = y.shape[-1], y.numel(), y.dtype, _io_dtype(y), _F32
    if n == 0:
        raise ValueError("y must not be empty")
    rows = n // D
    if out_dtype is None:
        out_dtype = (residual if residual is not None else out if out is not None else y).dtype
    if group is None:
        group = D if w is None else w.numel()
    st_y, st_out, st_h = _rows(y, rows, D, dt, dev, "y"), D, D
    if h is not None:
        if w_next is None:
            raise ValueError("h needs w_next")
        st_h = _rows(h, rows, D, dt, dev, "h")
    elif w_next is not None:
        h = torch.empty_like(y, memory_format=torch.contiguous_format)
    if out is None:
        out = torch.empty_like(y, dtype=out_dtype, memory_format=torch.contiguous_format)
    else:
        st_out = _rows(out, rows, D, out_dtype, dev, "out")
    rc = (_lib or library()).block_norm_forward(
        y.data_ptr(), _dense(w, (group,), f32, dev, "w"), None if gate is None else gate.data_ptr(),
        None if residual is None else residual.data_ptr(),
        _dense(scale, (D,), f32, dev, "scale"), _dense(w_next, (D,), f32, dev, "w_next"), rows, D,
        group, io, _io_dtype(out), gate_act, eps,
        _pack_norm_strides(
            st_y,
            0 if gate is None else _rows(gate, rows, D, dt, dev, "gate"),
            0 if residual is None else _rows(residual, rows, D, out_dtype, dev, "residual"),
            st_out, st_h),
        out.data_ptr(), None if h is None else h.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "block_norm_forward")
    return out, h


# ---------------------------------------------------------------- fixed-state mixers
# Made once per layer and decoded token too: arguments travel as one packed record.
_RECORDS = tuple(struct.Struct(x) for x in ("@10P12q10if", "@13PNP12q8i", "@8P4q7i"))
_pack_window, _pack_scan, _pack_conv = (x.pack for x in _RECORDS)
_I32 = torch.int32


def _elsewhere_needed(t, stream):
    """Whether the call has to be made under another current device or stream."""
    if not t.is_cuda:
        raise ValueError("tensors passed to the CUDA path must be on a CUDA device")
    return stream is not None or t.get_device() != _current_device()


def _addr(t, shape, dtype, dev, what):
    """Address of a contiguous tensor of this shape, or 0 for None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        _want(t, shape, dtype, dev, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _starts(seq_starts, B, dev):
    """(address, number of sequences) of packed sequences' bounds."""
    if seq_starts is None:
        return 0, B
    if B != 1:
        raise ValueError("seq_starts needs B = 1")
    n_seq = seq_starts.numel() - 1
    if n_seq < 1:
        raise ValueError("seq_starts must be a contiguous vector of n_seq + 1 entries")
    return _addr(seq_starts, (n_seq + 1,), _I32, dev, "seq_starts"), n_seq


def _caches(cache_k, cache_v, Hk, places, d, dt, dev):
    """(number of slots, addresses) of a pair of window-attention caches."""
    if cache_k is None or cache_v is None:
        if cache_k is not cache_v:
            raise ValueError("cache_k and cache_v are given together")
        return 0, 0, 0
    if cache_k.dim() != 4:
        raise ValueError("cache_k must have four dimensions")
    shape = (cache_k.shape[0], Hk, places, d)
    return (shape[0], _addr(cache_k, shape, dt, dev, "cache_k"),
            _addr(cache_v, shape, dt, dev, "cache_v"))


def window_attention_forward(q, k, v, window: int, sinks: int = 0,
                             scale: Optional[float] = None,
                             cache_k: Optional[torch.Tensor] = None,
                             cache_v: Optional[torch.Tensor] = None,
                             slots: Optional[torch.Tensor] = None,
                             past: Optional[torch.Tensor] = None,
                             seq_starts: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None, stream=None):
    """Causal attention with a sliding window over whole sequences, whose first
    ``sinks`` tokens stay visible (see ``window_attention_forward`` in
    include/ttt_mixers.h).

    q [B, Hq, N, d], k, v [B, Hk, N, d], bf16 or fp32, any strides with the
    last dimension contiguous.  cache_k, cache_v [n_slots, Hk, sinks + window, d]
    of the same type, contiguous, updated in place: the keys and values that
    ``window_attention_step`` and later turns read.  slots int32 [n_seq or B]
    (negative: no cache) or None; past int32 [n_seq or B], the tokens already in
    the caches, or None.  seq_starts: int32 [n_seq + 1] for sequences packed along
    the token axis (B = 1).  scale: d ** -0.5 when None.  Without ``out``, the
    outputs are stored in q's order of dimensions.  Returns out [B, Hq, N, d].
    """
    if _elsewhere_needed(q, stream):
        with _elsewhere(q.device, stream):
            return window_attention_forward(q, k, v, window, sinks, scale, cache_k, cache_v, slots,
                                            past, seq_starts, out)
    dev, dt, io = q.device, q.dtype, _io_dtype(q)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must have four dimensions")
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    shape = (B, Hk, N, d)
    _want(k, shape, dt, dev, "k")
    _want(v, shape, dt, dev, "v")
    starts, n_seq = _starts(seq_starts, B, dev)
    n_slots, ck, cv = _caches(cache_k, cache_v, Hk, sinks + window, d, dt, dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, (B, Hq, N, d), dt, dev, "out")
    rc = (_lib or library()).ttt_binding_window_forward(_pack_window(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), ck, cv,
        _addr(slots, (n_seq,), _I32, dev, "slots"), _addr(past, (n_seq,), _I32, dev, "past"), starts,
        out.data_ptr(), _raw_stream(dev.index), *_strides(q, "q")[:3], *_strides(k, "k")[:3],
        *_strides(v, "v")[:3], *_strides(out, "out")[:3], n_slots, n_seq, B, Hq, Hk, N, d, window,
        sinks, io, d ** -0.5 if scale is None else scale))
    if rc:
        _check(rc, "window_attention_forward")
    return out


def window_attention_step(q, k, v, cache_k, cache_v, positions, window: int, sinks: int = 0,
                          slots: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, stream=None):
    """One token of each of B sequences: its key and value are put into the
    cache, and it attends to what the cache then holds (see
    ``window_attention_step`` in include/ttt_mixers.h).

    q [B, Hq, d], k, v [B, Hk, d], bf16 or fp32, last dimension contiguous;
    cache_k, cache_v [n_slots, Hk, sinks + window, d] of the same type; positions
    int32 [B], the number of tokens before; slots int32 [B] (negative: an idle
    row) or None.  Returns out [B, Hq, d].
    """
    if _elsewhere_needed(q, stream):
        with _elsewhere(q.device, stream):
            return window_attention_step(q, k, v, cache_k, cache_v, positions, window, sinks, slots,
                                         scale, out)
    dev, dt, io = q.device, q.dtype, _io_dtype(q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must have three dimensions")
    B, Hq, d = q.shape
    Hk = k.shape[1]
    shape = (B, Hk, d)
    _want(k, shape, dt, dev, "k")
    _want(v, shape, dt, dev, "v")
    n_slots, ck, cv = _caches(cache_k, cache_v, Hk, sinks + window, d, dt, dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, (B, Hq, d), dt, dev, "out")
    rc = (_lib or library()).ttt_binding_window_step(_pack_window(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), ck, cv, _addr(slots, (B,), _I32, dev, "slots"),
        _addr(positions, (B,), _I32, dev, "positions"), 0, out.data_ptr(), _raw_stream(dev.index),
        *_strides(q, "q")[:2], 0, *_strides(k, "k")[:2], 0, *_strides(v, "v")[:2], 0,
        *_strides(out, "out")[:2], 0, n_slots, B, B, Hq, Hk, 1, d, window, sinks, io,
        d ** -0.5 if scale is None else scale))
    if rc:
        _check(rc, "window_attention_step")
    return out


def _groups(t, shape, dtype, dev, what):
    """Strides of a [rows.., G, S] tensor whose tokens are contiguous."""
    _want(t, shape, dtype, dev, what)
    st = t.stride()
    if (shape[-1] > 1 and st[-1] != 1) or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{what} must be contiguous in its last two dimensions")
    return st[:-2]


def selective_scan_workspace_size(B, N, D, S, G, n_seq, io_dtype) -> int:
    return library().selective_scan_workspace_size(B, N, D, S, G, n_seq, io_dtype)


_scan_need = functools.lru_cache(maxsize=4096)(selective_scan_workspace_size)   # by sizes alone


def selective_scan_forward(x, dt, A, B, C, D: Optional[torch.Tensor] = None,
                           dt_bias: Optional[torch.Tensor] = None,
                           z: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                           state: Optional[torch.Tensor] = None,
                           seq_starts: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None,
                           state_out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """The selective state space scan over whole sequences (see
    ``selective_scan_forward`` in include/ttt_mixers.h).

    x, dt, z [batch, N, channels], bf16 or fp32, any strides with the last dimension
    contiguous; A [channels, S] fp32; B, C [batch, N, G, S] in x's type, a token's
    numbers contiguous; D, dt_bias [channels] fp32 or None; state fp32
    [n_seq or batch, channels, S] or None (zeros).  seq_starts: int32 [n_seq + 1]
    for sequences packed along the token axis (batch of 1).  Returns (out
    [batch, N, channels], state_out [n_seq or batch, channels, S]).
    """
    if _elsewhere_needed(x, stream):
        with _elsewhere(x.device, stream):
            return selective_scan_forward(x, dt, A, B, C, D, dt_bias, z, dt_softplus, state,
                                          seq_starts, out, state_out, workspace)
    if x.dim() != 3 or B.dim() != 4:
        raise ValueError("x must have three dimensions, B four")
    dev, ty, io, f32, shape = x.device, x.dtype, _io_dtype(x), _F32, x.shape
    nb, N, ch = shape
    bc = B.shape
    G, S = bc[2:]
    _want(dt, shape, ty, dev, "dt")
    if z is not None:
        _want(z, shape, ty, dev, "z")
    if bc[:2] != (nb, N):
        raise ValueError(f"B must hold {nb} x {N} tokens, got shape {tuple(bc)}")
    sb, sc = _groups(B, bc, ty, dev, "B"), _groups(C, bc, ty, dev, "C")
    starts, n_seq = _starts(seq_starts, nb, dev)
    states = (n_seq, ch, S)
    if out is None:
        out = torch.empty_like(x)   # x's order of dimensions
    else:
        _want(out, shape, ty, dev, "out")
    if state_out is None:
        state_out = A.new_empty(states)
    if workspace is None:
        workspace = torch.empty(max(_scan_need(nb, N, ch, S, G, n_seq, io), 256), device=dev,
                                dtype=torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    rc = (_lib or library()).ttt_binding_scan_forward(_pack_scan(
        x.data_ptr(), dt.data_ptr(), _addr(A, (ch, S), f32, dev, "A"), B.data_ptr(), C.data_ptr(),
        _addr(D, (ch,), f32, dev, "D"), _addr(dt_bias, (ch,), f32, dev, "dt_bias"),
        0 if z is None else z.data_ptr(), _addr(state, states, f32, dev, "state"), starts,
        out.data_ptr(), _addr(state_out, states, f32, dev, "state_out"), workspace.data_ptr(),
        workspace.nbytes, _raw_stream(dev.index), *_strides(x, "x")[:2], *_strides(dt, "dt")[:2],
        *((0, 0) if z is None else _strides(z, "z")[:2]), *sb, *sc, *_strides(out, "out")[:2], n_seq,
        nb, N, ch, S, G, io, 1 if dt_softplus else 0))
    if rc:
        _check(rc, "selective_scan_forward")
    return out, state_out


def selective_scan_step(x, dt, A, B, C, state, D: Optional[torch.Tensor] = None,
                        dt_bias: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                        slots: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, stream=None):
    """The selective state space scan for one token of each row, on a pool of
    states that is updated in place (see ``selective_scan_step`` in
    include/ttt_mixers.h).

    x, dt, z [rows, channels], B, C [rows, G, S]; state [n_slots, channels, S]
    fp32; slots int32 [rows] (negative: an idle row) or None.  The others as for
    ``selective_scan_forward``.  Returns out [rows, channels].
    """
    if _elsewhere_needed(x, stream):
        with _elsewhere(x.device, stream):
            return selective_scan_step(x, dt, A, B, C, state, D, dt_bias, z, dt_softplus, slots, out)
    if x.dim() != 2 or B.dim() != 3 or state.dim() != 3:
        raise ValueError("x must have two dimensions, B and state three")
    dev, ty, io, f32, shape = x.device, x.dtype, _io_dtype(x), _F32, x.shape
    nb, ch = shape
    bc = B.shape
    G, S = bc[1:]
    _want(dt, shape, ty, dev, "dt")
    if z is not None:
        _want(z, shape, ty, dev, "z")
    if bc[0] != nb:
        raise ValueError(f"B must hold {nb} rows, got shape {tuple(bc)}")
    (sb,), (sc,) = _groups(B, bc, ty, dev, "B"), _groups(C, bc, ty, dev, "C")
    n_slots = state.shape[0]
    if out is None:
        out = torch.empty_like(x)
    else:
        _want(out, shape, ty, dev, "out")
    rc = (_lib or library()).ttt_binding_scan_step(_pack_scan(
        x.data_ptr(), dt.data_ptr(), _addr(A, (ch, S), f32, dev, "A"), B.data_ptr(), C.data_ptr(),
        _addr(D, (ch,), f32, dev, "D"), _addr(dt_bias, (ch,), f32, dev, "dt_bias"),
        0 if z is None else z.data_ptr(), 0, _addr(slots, (nb,), _I32, dev, "slots"), out.data_ptr(),
        _addr(state, (n_slots, ch, S), f32, dev, "state"), 0, 0, _raw_stream(dev.index),
        _strides(x, "x")[0], 0, _strides(dt, "dt")[0], 0, 0 if z is None else _strides(z, "z")[0], 0,
        sb, 0, sc, 0, _strides(out, "out")[0], 0, n_slots, nb, 1, ch, S, G, io,
        1 if dt_softplus else 0))
    if rc:
        _check(rc, "selective_scan_step")
    return out


def short_conv_forward(x, w, bias: Optional[torch.Tensor] = None, silu: bool = False,
                       state: Optional[torch.Tensor] = None,
                       seq_starts: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       state_out: Optional[torch.Tensor] = None, stream=None):
    """The short causal convolution of each channel over whole sequences (see
    ``short_conv_forward`` in include/ttt_mixers.h).

    x [B, N, D], bf16 or fp32, any strides with the last dimension contiguous;
    w [D, W] fp32 (w[:, W - 1] meets the token itself); bias [D] fp32 or None;
    state [n_seq or B, W - 1, D] in x's type, the inputs before each sequence,
    oldest first, or None (zeros).  seq_starts: int32 [n_seq + 1] for sequences
    packed along the token axis (B = 1).  Returns (out [B, N, D], state_out).
    """
    if _elsewhere_needed(x, stream):
        with _elsewhere(x.device, stream):
            return short_conv_forward(x, w, bias, silu, state, seq_starts, out, state_out)
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must have three dimensions, w two")
    dev, ty, io, shape = x.device, x.dtype, _io_dtype(x), x.shape
    B, N, D = shape
    W = w.shape[1]
    starts, n_seq = _starts(seq_starts, B, dev)
    rows = (n_seq, max(W - 1, 0), D)
    if out is None:
        out = torch.empty_like(x)   # x's order of dimensions
    else:
        _want(out, shape, ty, dev, "out")
    if state_out is None:
        state_out = x.new_empty(rows)
    rc = (_lib or library()).ttt_binding_conv_forward(_pack_conv(
        x.data_ptr(), _addr(w, (D, W), _F32, dev, "w"), _addr(bias, (D,), _F32, dev, "bias"),
        _addr(state, rows, ty, dev, "state"), starts, out.data_ptr(),
        _addr(state_out, rows, ty, dev, "state_out"), _raw_stream(dev.index), *_strides(x, "x")[:2],
        *_strides(out, "out")[:2], n_seq, B, N, D, W, io, 1 if silu else 0))
    if rc:
        _check(rc, "short_conv_forward")
    return out, state_out


def short_conv_step(x, w, state, bias: Optional[torch.Tensor] = None, silu: bool = False,
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream=None):
    """The short causal convolution for one token of each row, on a pool of
    states that is updated in place (see ``short_conv_step`` in
    include/ttt_mixers.h).

    x [B, D]; w [D, W] fp32; state [n_slots, W - 1, D] in x's type; slots int32
    [B] (negative: an idle row) or None.  Returns out [B, D].
    """
    if _elsewhere_needed(x, stream):
        with _elsewhere(x.device, stream):
            return short_conv_step(x, w, state, bias, silu, slots, out)
    if x.dim() != 2 or w.dim() != 2 or state.dim() != 3:
        raise ValueError("x and w must have two dimensions, state three")
    dev, ty, io, shape = x.device, x.dtype, _io_dtype(x), x.shape
    B, D = shape
    W, n_slots = w.shape[1], state.shape[0]
    if out is None:
        out = torch.empty_like(x)
    else:
        _want(out, shape, ty, dev, "out")
    rc = (_lib or library()).ttt_binding_conv_step(_pack_conv(
        x.data_ptr(), _addr(w, (D, W), _F32, dev, "w"), _addr(bias, (D,), _F32, dev, "bias"), 0,
        _addr(slots, (B,), _I32, dev, "slots"), out.data_ptr(),
        _addr(state, (n_slots, max(W - 1, 0), D), ty, dev, "state"), _raw_stream(dev.index),
        _strides(x, "x")[0], 0, _strides(out, "out")[0], 0, n_slots, B, 1, D, W, io,
        1 if silu else 0))
    if rc:
        _check(rc, "short_conv_step")
    return out


def device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return library().ttt_device_status(_stream(stream))


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(library().ttt_launch_count())


def profile_start():
    library().ttt_profile_start()


def profile_stop():
    """Per launch kind: dict(name, kernel, launches, ms, flops, bytes, sm_ms)."""
    arr = (ProfileEntry * 64)()
    n = library().ttt_profile_stop(arr, 64)
    if n < 0:
        raise TTTError(n, "ttt_profile_stop")
    return [dict(name=e.name.decode(), kernel=e.kernel.decode(), launches=e.launches, ms=e.ms,
                 flops=e.flops, bytes=e.bytes, sm_ms=e.sm_ms) for e in arr[:n]]


def set_wait_limit_ns(ns: int):
    library().ttt_set_wait_limit_ns(int(ns))


def selftest_withhold_release(bh: int):
    """Test hook: from the next linear-attention call on, batch-head ``bh``'s
    state items never report completion, so the items waiting for them run
    into their bounded waits (-1 turns it off).  See include/ttt_selftest.h."""
    library().ttt_selftest_withhold_release(int(bh))


def selftest_withhold_delta(kernel: int):
    """Test hook: from the next delta-rule call on, a wait of one of the chunk
    form's kernels runs out (0 turns it off).  See include/ttt_selftest.h."""
    library().ttt_selftest_withhold_delta(int(kernel))


def selftest_withhold_window(what: int):
    """Test hook: from the next call on, a wait of the window attention's tensor-core
    kernel runs out (0 turns it off).  See include/ttt_selftest.h."""
    library().ttt_selftest_withhold_window(int(what))


def selftest_gemm(A, B, a_mn_major: bool, b_mn_major: bool, tile_n: int = 128, stream=None):
    """fp32 D = A * B through the library's GEMM building block (self-test).

    A: [Z, M, K] (or [Z, K, M] when a_mn_major); B: [Z, N, K] (or [Z, K, N]).
    """
    lib = library()
    Z = A.shape[0]
    if a_mn_major:
        K, M = A.shape[1], A.shape[2]
    else:
        M, K = A.shape[1], A.shape[2]
    N = B.shape[2] if b_mn_major else B.shape[1]
    D = torch.empty((Z, M, N), device=A.device, dtype=torch.float32)
    rc = lib.ttt_selftest_gemm(_ptr(A), _ptr(B), _ptr(D), Z, M, N, K, int(a_mn_major),
                               int(b_mn_major), _io_dtype(A), tile_n, _stream(stream))
    _check(rc, "ttt_selftest_gemm")
    return D
