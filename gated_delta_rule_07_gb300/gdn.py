"""ctypes binding of libgdn.so (the C ABI declared in include/gdn.h).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  Functions named after the C entry points take torch CUDA tensors, pass their
data pointers and the current torch stream, and raise ``GdnError`` on a non-OK status.
``forward()`` is the convenience call that allocates the outputs and the workspace.

Importing this module loads the library and raises ImportError when it has not been built
(``python -m gated_delta_rule_07_gb300.build``); there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

LIB_PATH = _build.LIB

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libgdn.so is not built ({LIB_PATH}); run "
                      "`python -m gated_delta_rule_07_gb300.build` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)

GDN_OK = 0
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARGUMENT", 2: "GDN_ERR_UNSUPPORTED",
                3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_CUDA", 5: "GDN_ERR_DEVICE_TIMEOUT",
                6: "GDN_ERR_DEVICE_INPUT", 7: "GDN_ERR_DEVICE_RANGE"}
GDN_BF16, GDN_F32 = 0, 1
EXPORTED = ("gdn_status_string", "gdn_check_problem", "gdn_workspace_size", "gdn_forward",
            "gdn_chunk_prepare", "gdn_segment_summary", "gdn_state_prefix_scan",
            "gdn_chunk_emit", "gdn_device_status", "gdn_version",
            "gdn_segment_summary_fused", "gdn_chunk_emit_fused", "gdn_last_error_string",
            "gdn_forward_static_scratch", "gdn_forward_timed", "gdn_forward_with_limits",
            "gdn_check_decode_problem", "gdn_decode_step", "gdn_backward_workspace_size",
            "gdn_backward", "gdn_prologue", "gdn_qk_norm_rope",
            "gdn_qk_norm_rope_backward_workspace_size", "gdn_qk_norm_rope_backward",
            "gdn_kv_append", "gdn_kv_read", "gdn_kv_attention_workspace_size",
            "gdn_kv_attention")


class Problem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("hk", ctypes.c_int32), ("hv", ctypes.c_int32), ("k_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("segments_per_seq", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


class DecodeProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("slots", ctypes.c_int32), ("hk", ctypes.c_int32),
                ("hv", ctypes.c_int32), ("k_dim", ctypes.c_int32), ("v_dim", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


class PrologueProblem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("hk", ctypes.c_int32), ("hv", ctypes.c_int32), ("k_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("conv_width", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


class QkRopeProblem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("hq", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("style", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("max_positions", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class KvProblem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("hq", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {gdn_status_string(status)}"
        if status == 4:
            msg += f" ({_lib.gdn_last_error_string().decode()})"
        super().__init__(msg)


_vp, _fp, _ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_pp = ctypes.POINTER(Problem)
_lib.gdn_status_string.restype = ctypes.c_char_p
_lib.gdn_status_string.argtypes = [ctypes.c_int]
_lib.gdn_last_error_string.restype = ctypes.c_char_p
_lib.gdn_last_error_string.argtypes = []
_lib.gdn_check_problem.argtypes = [_pp]
_lib.gdn_workspace_size.restype = ctypes.c_size_t
_lib.gdn_workspace_size.argtypes = [_pp]
_lib.gdn_forward.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _vp,
                             ctypes.c_size_t, _vp]
_lib.gdn_forward_timed.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _vp,
                             ctypes.c_size_t, _vp, ctypes.POINTER(ctypes.c_float)]
_lib.gdn_forward_with_limits.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _vp,
                                         ctypes.c_size_t, _vp, ctypes.c_longlong, ctypes.c_int]
_lib.gdn_chunk_prepare.argtypes = [_pp, _vp, _vp, _fp, _fp, _ip, _vp, _vp, _fp, _ip, _vp]
_lib.gdn_segment_summary.argtypes = [_pp, _vp, _vp, _vp, _fp, _ip, _fp, _fp, _ip, _vp]
_lib.gdn_state_prefix_scan.argtypes = [_pp, _fp, _fp, _fp, _fp, _fp, _vp]
_lib.gdn_chunk_emit.argtypes = [_pp, _vp, _vp, _vp, _vp, _fp, _fp, _ip, _vp, _fp, _ip, _vp]
_lib.gdn_device_status.argtypes = [_vp, ctypes.c_int, _vp]
_lib.gdn_segment_summary_fused.argtypes = [_pp, _vp, _vp, _fp, _fp, _ip, _fp, _fp, ctypes.c_int,
                                           _ip, _vp]
_lib.gdn_chunk_emit_fused.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _ip, _vp]
_lib.gdn_forward_static_scratch.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _vp]
_lib.gdn_backward_workspace_size.restype = ctypes.c_size_t
_lib.gdn_backward_workspace_size.argtypes = [_pp]
_lib.gdn_backward.argtypes = [_pp, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _fp, _vp, _vp, _vp,
                              _fp, _fp, _fp, _vp, ctypes.c_size_t, _vp]
_lib.gdn_prologue.argtypes = [ctypes.POINTER(PrologueProblem), _vp, _fp, _vp, _vp, _vp, _fp, _fp,
                              _ip, _vp, _vp, _vp, _fp, _fp, _vp, _ip, _vp]
_dpp = ctypes.POINTER(DecodeProblem)
_lib.gdn_check_decode_problem.argtypes = [_dpp]
_lib.gdn_decode_step.argtypes = [_dpp, _vp, _vp, _vp, _fp, _fp, _ip, _fp, _vp, _ip, _vp]
_rp = ctypes.POINTER(QkRopeProblem)
_lib.gdn_qk_norm_rope.argtypes = [_rp, _vp, _vp, _ip, _fp, _fp, _fp, _vp, _vp, _ip, _vp]
_lib.gdn_qk_norm_rope_backward_workspace_size.restype = ctypes.c_size_t
_lib.gdn_qk_norm_rope_backward_workspace_size.argtypes = [_rp]
_lib.gdn_qk_norm_rope_backward.argtypes = [_rp, _vp, _vp, _ip, _fp, _fp, _fp, _vp, _vp, _vp, _vp,
                                           _fp, _fp, _vp, ctypes.c_size_t, _ip, _vp]
_cp, _kp = ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvProblem)
_lib.gdn_kv_append.argtypes = [_cp, _kp, _vp, _vp, _ip, _ip, _ip, _ip, _vp]
_lib.gdn_kv_read.argtypes = [_cp, _kp, _ip, _ip, _ip, _vp, _vp, _ip, _vp]
_lib.gdn_kv_attention_workspace_size.restype = ctypes.c_size_t
_lib.gdn_kv_attention_workspace_size.argtypes = [_cp, _kp]
_lib.gdn_kv_attention.argtypes = [_cp, _kp, _vp, _ip, _ip, _ip, ctypes.c_float, ctypes.c_int32,
                                  _vp, _fp, _vp, ctypes.c_size_t, _ip, _vp]
for _n in EXPORTED:
    if _n not in ("gdn_status_string", "gdn_workspace_size", "gdn_last_error_string",
                  "gdn_backward_workspace_size", "gdn_qk_norm_rope_backward_workspace_size",
                  "gdn_kv_attention_workspace_size"):
        getattr(_lib, _n).restype = ctypes.c_int


def gdn_status_string(status: int) -> str:
    return _lib.gdn_status_string(int(status)).decode()


def gdn_version() -> int:
    return _lib.gdn_version()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # (what torch.cuda.current_stream().cuda_stream gives, without its object)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status, where):
    if status != GDN_OK:
        raise GdnError(status, where)


def make_problem(T, N, hk, hv, K, V, P=1, dtype=torch.bfloat16, chunk=64):
    io = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}.get(dtype)
    if io is None:
        raise GdnError(2, f"dtype {dtype}")
    return Problem(int(T), int(N), int(hk), int(hv), int(K), int(V), int(chunk), int(P), io)


def problem_for(q, v, cu_seqlens=None, P=1) -> Problem:
    T, hk, K = q.shape
    hv, V = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    return make_problem(T, N, hk, hv, K, V, P, q.dtype)


def gdn_check_problem(p: Problem) -> int:
    return _lib.gdn_check_problem(ctypes.byref(p))


def gdn_workspace_size(p: Problem) -> int:
    return int(_lib.gdn_workspace_size(ctypes.byref(p)))


def gdn_forward(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace, ws_bytes=None,
                stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_forward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                            _ptr(h0), _ptr(cu_seqlens), _ptr(out), _ptr(h_final),
                            _ptr(workspace), int(ws_bytes), _stream(stream)), "gdn_forward")


def gdn_forward_timed(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace,
                      ws_bytes=None, stream=None):
    """gdn_forward that waits for its own end and returns the milliseconds of (summaries,
    prefix scan, phase 3, first summary kernel) measured with CUDA events on the stream."""
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    ms = (ctypes.c_float * 4)()
    _check(_lib.gdn_forward_timed(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(h0), _ptr(cu_seqlens), _ptr(out), _ptr(h_final),
                                  _ptr(workspace), int(ws_bytes), _stream(stream), ms),
           "gdn_forward_timed")
    return float(ms[0]), float(ms[1]), float(ms[2]), float(ms[3])


def gdn_forward_with_limits(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace,
                            wait_cycles=0, fault=0, ws_bytes=None, stream=None):
    """gdn_forward with a given limit on the device's bounded waits and an optional injected
    fault (tests of the failure detection; see include/gdn.h)."""
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_forward_with_limits(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                        _ptr(beta), _ptr(h0), _ptr(cu_seqlens), _ptr(out),
                                        _ptr(h_final), _ptr(workspace), int(ws_bytes),
                                        _stream(stream), int(wait_cycles), int(fault)),
           "gdn_forward_with_limits")


def gdn_forward_static_scratch(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, stream=None):
    """gdn_forward without a workspace: for callers that cannot allocate device memory.  Its
    scratch is the library's own 64 MiB device array (see include/gdn.h for the limits)."""
    _check(_lib.gdn_forward_static_scratch(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                           _ptr(beta), _ptr(h0), _ptr(cu_seqlens), _ptr(out),
                                           _ptr(h_final), _stream(stream)),
           "gdn_forward_static_scratch")


def gdn_chunk_prepare(p, k, v, g, beta, cu_seqlens, w, u, gcum, dev_status=None, stream=None):
    _check(_lib.gdn_chunk_prepare(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(cu_seqlens), _ptr(w), _ptr(u), _ptr(gcum),
                                  _ptr(dev_status), _stream(stream)), "gdn_chunk_prepare")


def gdn_segment_summary(p, k, w, u, gcum, cu_seqlens, M, U, dev_status=None, stream=None):
    _check(_lib.gdn_segment_summary(ctypes.byref(p), _ptr(k), _ptr(w), _ptr(u), _ptr(gcum),
                                    _ptr(cu_seqlens), _ptr(M), _ptr(U), _ptr(dev_status),
                                    _stream(stream)), "gdn_segment_summary")


def gdn_state_prefix_scan(p, M, U, h0, h_in, h_final, stream=None):
    _check(_lib.gdn_state_prefix_scan(ctypes.byref(p), _ptr(M), _ptr(U), _ptr(h0), _ptr(h_in),
                                      _ptr(h_final), _stream(stream)), "gdn_state_prefix_scan")


def gdn_chunk_emit(p, q, k, w, u, gcum, h_in, cu_seqlens, out, h_final, dev_status=None,
                   stream=None):
    _check(_lib.gdn_chunk_emit(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(w), _ptr(u), _ptr(gcum),
                               _ptr(h_in), _ptr(cu_seqlens), _ptr(out), _ptr(h_final),
                               _ptr(dev_status), _stream(stream)), "gdn_chunk_emit")


def gdn_segment_summary_fused(p, k, v, g, beta, cu_seqlens, M, U, skip_last=False,
                              dev_status=None, stream=None):
    _check(_lib.gdn_segment_summary_fused(ctypes.byref(p), _ptr(k), _ptr(v), _ptr(g),
                                          _ptr(beta), _ptr(cu_seqlens), _ptr(M), _ptr(U),
                                          int(bool(skip_last)), _ptr(dev_status),
                                          _stream(stream)), "gdn_segment_summary_fused")


def gdn_chunk_emit_fused(p, q, k, v, g, beta, h_in, cu_seqlens, out, h_final, dev_status=None,
                         stream=None):
    _check(_lib.gdn_chunk_emit_fused(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                     _ptr(beta), _ptr(h_in), _ptr(cu_seqlens), _ptr(out),
                                     _ptr(h_final), _ptr(dev_status), _stream(stream)),
           "gdn_chunk_emit_fused")


def gdn_backward_workspace_size(p: Problem) -> int:
    return int(_lib.gdn_backward_workspace_size(ctypes.byref(p)))


def gdn_backward(p, q, k, v, g, beta, h0, cu_seqlens, dout, dh_final, dq, dk, dv, dg, dbeta,
                 dh0, workspace, ws_bytes=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_backward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                             _ptr(h0), _ptr(cu_seqlens), _ptr(dout), _ptr(dh_final), _ptr(dq),
                             _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0),
                             _ptr(workspace), int(ws_bytes), _stream(stream)), "gdn_backward")


def backward(q, k, v, g, beta, dout, h0=None, dh_final=None, cu_seqlens=None, workspace=None,
             check_status=False, stream=None):
    """Gradients (dq, dk, dv, dg, dbeta, dh0) of <dout, out> + <dh_final, h_final> through the
    forward on the same inputs; allocates the outputs (and the workspace unless given)."""
    p = problem_for(q, v, cu_seqlens)
    N = p.num_seqs
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    dh0 = torch.empty(N, p.hv, p.k_dim, p.v_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(gdn_backward_workspace_size(p), 256), dtype=torch.uint8,
                                device=q.device)
    gdn_backward(p, q, k, v, g, beta, h0, cu_seqlens, dout, dh_final, dq, dk, dv, dg, dbeta,
                 dh0, workspace, stream=stream)
    if check_status:
        _check(gdn_device_status(workspace, True, stream), "gdn_backward (device status)")
    return dq, dk, dv, dg, dbeta, dh0


def gdn_prologue(p, x, conv_w, conv_state_in, a, b, A_log, dt_bias, cu_seqlens, q, k, v, g,
                 beta, conv_state_out, dev_status=None, stream=None):
    _check(_lib.gdn_prologue(ctypes.byref(p), _ptr(x), _ptr(conv_w), _ptr(conv_state_in), _ptr(a),
                             _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(cu_seqlens), _ptr(q),
                             _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(conv_state_out),
                             _ptr(dev_status), _stream(stream)), "gdn_prologue")


def prologue(x, conv_w, a, b, A_log, dt_bias, hk, hv, K, V, conv_state=None, cu_seqlens=None,
             activation="none", check_status=False, stream=None):
    """q, k, v, g, beta, new conv state from the projections (layouts of include/gdn.h)."""
    T = x.shape[0]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    W = conv_w.shape[1]
    io = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}[x.dtype]
    p = PrologueProblem(T, N, hk, hv, K, V, W, {"none": 0, "silu": 1}[activation], io)
    dev = x.device
    q = torch.empty(T, hk, K, dtype=x.dtype, device=dev)
    k = torch.empty_like(q)
    v = torch.empty(T, hv, V, dtype=x.dtype, device=dev)
    g = torch.empty(T, hv, dtype=torch.float32, device=dev)
    beta = torch.empty_like(g)
    new_state = torch.empty(N, x.shape[1], max(W - 1, 0), dtype=x.dtype, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev) if check_status else None
    gdn_prologue(p, x, conv_w, conv_state, a, b, A_log, dt_bias, cu_seqlens, q, k, v, g, beta,
                 new_state if W > 1 else None, st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "gdn_prologue (device status)")
    return q, k, v, g, beta, new_state


def make_decode_problem(B, slots, hk, hv, K, V, dtype=torch.bfloat16) -> DecodeProblem:
    io = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}.get(dtype)
    if io is None:
        raise GdnError(2, f"dtype {dtype}")
    return DecodeProblem(int(B), int(slots), int(hk), int(hv), int(K), int(V), io)


def decode_problem_for(q, v, state) -> DecodeProblem:
    B, hk, K = q.shape
    return make_decode_problem(B, state.shape[0], hk, v.shape[1], K, v.shape[2], q.dtype)


def gdn_check_decode_problem(p: DecodeProblem) -> int:
    return _lib.gdn_check_decode_problem(ctypes.byref(p))


def gdn_decode_step(p, q, k, v, g, beta, slot, state, out, dev_status=None, stream=None):
    _check(_lib.gdn_decode_step(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                _ptr(slot), _ptr(state), _ptr(out), _ptr(dev_status),
                                _stream(stream)), "gdn_decode_step")


def decode(q, k, v, g, beta, slot, state, out=None, check_status=False, stream=None):
    """One decode step: row b continues the request held in state[slot[b]] (updated in place).
    Returns out [B, hv, V]; with check_status, waits and raises on a device-side error."""
    p = decode_problem_for(q, v, state)
    if out is None:
        out = torch.empty_like(v)
    st = torch.zeros(1, dtype=torch.int32, device=q.device) if check_status else None
    gdn_decode_step(p, q, k, v, g, beta, slot, state, out, st, stream)
    if check_status:
        _check(gdn_device_status(st, reset=True, stream=stream), "gdn_decode_step (device status)")
    return out


def gdn_device_status(status_word, reset=True, stream=None) -> int:
    """Synchronous read of a device status word (a dev_status tensor or a workspace)."""
    return _lib.gdn_device_status(_ptr(status_word), int(bool(reset)), _stream(stream))


# ------------------------------------------------- softmax-attention layers' operators
#
# These calls are short on the GPU (a decode step's take a few microseconds), so the host's part
# is kept lean: each tensor is looked at once, in the order that costs least, and messages are
# only built for a refusal.

_IO = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_KV_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}
_ROPE_STYLES = {"half": 0, "pairs": 1}
_GDN_ERR_INVALID_ARGUMENT, _GDN_ERR_UNSUPPORTED = 1, 2
_F32, _I32 = torch.float32, torch.int32


def _refuse(where, why, status=_GDN_ERR_INVALID_ARGUMENT):
    raise GdnError(status, f"{where}: {why}")


def _io_of(where, t):
    io = _IO.get(t.dtype)
    if io is None:
        _refuse(where, f"dtype {t.dtype}", _GDN_ERR_UNSUPPORTED)
    return io


def _packed(where, name, t, shape, dtype):
    """t is a contiguous GPU tensor of this shape and dtype."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda:
        _refuse(where, f"{name} is to be a contiguous {dtype} tensor {tuple(shape)} on the GPU, "
                       f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _rows(where, name, t, dtype):
    """Shape, token and head stride of a [T, heads, D] GPU tensor whose last dimension is
    contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        _refuse(where, f"{name} is to be [tokens, heads, D] with a contiguous last dimension, "
                       f"got {tuple(shape)} with strides {stride}")
    if t.dtype is not dtype:
        _refuse(where, f"{name} is {t.dtype}, the call's dtype is {dtype}")
    if not t.is_cuda:
        _refuse(where, f"{name} is not on the GPU")
    return shape, stride[0], stride[1]


def _hold(stream, *tensors):
    """Temporaries and outputs allocated on the current stream and used on `stream`: their memory
    is not handed out again before the work on `stream` is done."""
    if hasattr(stream, "cuda_stream"):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _opt(t):
    return None if t is None else t.data_ptr()


def _rope_problem(where, q, k, positions, cos_sin, q_weight, k_weight, eps, weight_offset, style):
    io, dtype = _io_of(where, q), q.dtype
    (T, hq, D), qt, qh = _rows(where, "q", q, dtype)
    kshape, kt, kh = _rows(where, "k", k, dtype)
    if kshape[0] != T or kshape[2] != D:
        _refuse(where, f"q {tuple(q.shape)} and k {tuple(kshape)} do not go together")
    _packed(where, "positions", positions, (T,), _I32)
    tshape = cos_sin.shape
    if len(tshape) != 2:
        _refuse(where, "cos_sin is to be [positions, R]")
    _packed(where, "cos_sin", cos_sin, tshape, _F32)
    if q_weight is not None:
        _packed(where, "q_weight", q_weight, (D,), _F32)
    if k_weight is not None:
        _packed(where, "k_weight", k_weight, (D,), _F32)
    which = _ROPE_STYLES.get(style)
    if which is None:
        _refuse(where, f"style {style!r}")
    return QkRopeProblem(T, hq, kshape[1], D, tshape[1], which, io, tshape[0], eps,
                         weight_offset, qt, qh, kt, kh)


def gdn_qk_norm_rope(p, q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out,
                     dev_status=None, stream=None):
    _check(_lib.gdn_qk_norm_rope(p, q.data_ptr(), k.data_ptr(), positions.data_ptr(),
                                 cos_sin.data_ptr(), _opt(q_weight), _opt(k_weight),
                                 q_out.data_ptr(), k_out.data_ptr(), _opt(dev_status),
                                 _stream(stream)), "gdn_qk_norm_rope")


def qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, style="half", check_status=False, stream=None):
    """Queries [T, hq, D] and keys [T, hkv, D], normalised per head and rotated by position (see
    include/gdn.h); q and k may be slices of one projection.  Returns contiguous tensors."""
    p = _rope_problem("qk_norm_rope", q, k, positions, cos_sin, q_weight, k_weight, eps,
                      weight_offset, style)
    device, dtype = q.device, q.dtype
    q_out = torch.empty(q.shape, dtype=dtype, device=device)
    k_out = torch.empty(k.shape, dtype=dtype, device=device)
    st = torch.zeros(1, dtype=_I32, device=device) if check_status else None
    if stream is not None:
        _hold(stream, q_out, k_out, st)
    gdn_qk_norm_rope(p, q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out, st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "qk_norm_rope (device status)")
    return q_out, k_out


def gdn_qk_norm_rope_backward_workspace_size(p) -> int:
    return _lib.gdn_qk_norm_rope_backward_workspace_size(p)


def gdn_qk_norm_rope_backward(p, q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out,
                              dq, dk, dq_weight, dk_weight, workspace, ws_bytes=None,
                              dev_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_qk_norm_rope_backward(
        p, q.data_ptr(), k.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), _opt(q_weight),
        _opt(k_weight), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
        dq_weight.data_ptr(), dk_weight.data_ptr(), workspace.data_ptr(), ws_bytes,
        _opt(dev_status), _stream(stream)), "gdn_qk_norm_rope_backward")


def qk_norm_rope_backward(q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out, eps=1e-6,
                          weight_offset=0.0, style="half", workspace=None, check_status=False,
                          stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of <dq_out, q_out> + <dk_out, k_out> through
    qk_norm_rope on the same inputs."""
    where = "qk_norm_rope_backward"
    p = _rope_problem(where, q, k, positions, cos_sin, q_weight, k_weight, eps, weight_offset,
                      style)
    device, D = q.device, p.head_dim
    _packed(where, "dq_out", dq_out, q.shape, q.dtype)
    _packed(where, "dk_out", dk_out, k.shape, q.dtype)
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    dqw = torch.empty(D, dtype=_F32, device=device)
    dkw = torch.empty(D, dtype=_F32, device=device)
    if workspace is None:
        workspace = torch.empty(gdn_qk_norm_rope_backward_workspace_size(p), dtype=torch.uint8,
                                device=device)
    st = torch.zeros(1, dtype=_I32, device=device) if check_status else None
    if stream is not None:
        _hold(stream, dq, dk, dqw, dkw, workspace, st)
    gdn_qk_norm_rope_backward(p, q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out,
                              dq, dk, dqw, dkw, workspace, None, st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "qk_norm_rope_backward (device status)")
    return dq, dk, dqw, dkw


class KVCache:
    """The buffers of a paged 8-bit key/value cache (layouts of include/gdn.h):
    k [pages, hkv, page, D] and v [pages, hkv, page // 4, D, 4], both int8 or float8_e4m3fn;
    k_scale, v_scale [pages, hkv] fp32.  ``KVCache.empty`` allocates them."""

    def __init__(self, k, v, k_scale, v_scale):
        where = "KVCache"
        if k.dtype not in _KV_FORMATS:
            _refuse(where, f"dtype {k.dtype}", _GDN_ERR_UNSUPPORTED)
        if k.dim() != 4:
            _refuse(where, "k is to be [pages, hkv, page, D]")
        pages, hkv, page, D = k.shape
        _packed(where, "k", k, k.shape, k.dtype)
        _packed(where, "v", v, (pages, hkv, page // 4, D, 4), k.dtype)
        _packed(where, "k_scale", k_scale, (pages, hkv), _F32)
        _packed(where, "v_scale", v_scale, (pages, hkv), _F32)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.head_dim = hkv, D
        self.desc = KvCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), pages, page, hkv, D, _KV_FORMATS[k.dtype])

    @classmethod
    def empty(cls, pages, hkv, page, D, dtype=torch.int8, device="cuda"):
        """A cache of `pages` pages; nothing in it is initialised, or needs to be."""
        return cls(torch.empty(pages, hkv, page, D, dtype=dtype, device=device),
                   torch.empty(pages, hkv, page // 4, D, 4, dtype=dtype, device=device),
                   torch.empty(pages, hkv, dtype=_F32, device=device),
                   torch.empty(pages, hkv, dtype=_F32, device=device))


def _kv_sequences(where, T, block_table, lens, cu_seqlens):
    """Checks the tables of a cache call; the number of sequences and of pages in a table row."""
    shape = block_table.shape
    if len(shape) != 2:
        _refuse(where, "block_table is to be [sequences, pages]")
    _packed(where, "block_table", block_table, shape, _I32)
    N = shape[0]
    if lens is not None:
        _packed(where, "lengths", lens, (N,), _I32)
    if cu_seqlens is not None:
        _packed(where, "cu_seqlens", cu_seqlens, (N + 1,), _I32)
    elif N != 1 and N != T:
        _refuse(where, f"{T} rows of {N} sequences need cu_seqlens")
    return N, shape[1]


def gdn_kv_append(cache, p, k, v, block_table, ctx_lens, cu_seqlens, dev_status=None,
                  stream=None):
    _check(_lib.gdn_kv_append(cache, p, k.data_ptr(), v.data_ptr(), block_table.data_ptr(),
                              ctx_lens.data_ptr(), _opt(cu_seqlens), _opt(dev_status),
                              _stream(stream)), "gdn_kv_append")


def kv_append(cache, k, v, block_table, ctx_lens, cu_seqlens=None, check_status=False,
              stream=None):
    """Quantises new keys and values [T, hkv, D] into the cache's pages, behind the ctx_lens[n]
    tokens that each sequence already holds.  Without cu_seqlens the rows are one sequence's, or
    one row each of T sequences."""
    where = "kv_append"
    io, dtype = _io_of(where, k), k.dtype
    shape, kt, kh = _rows(where, "k", k, dtype)
    vshape, vt, vh = _rows(where, "v", v, dtype)
    T, h, D = shape
    if vshape != shape or h != cache.heads or D != cache.head_dim:
        _refuse(where, f"k {tuple(shape)} and v {tuple(vshape)} for a cache of {cache.heads} "
                       f"heads of {cache.head_dim}")
    N, max_pages = _kv_sequences(where, T, block_table, ctx_lens, cu_seqlens)
    p = KvProblem(T, N, max_pages, 0, io, kt, kh, vt, vh, 0, 0)
    st = torch.zeros(1, dtype=_I32, device=k.device) if check_status else None
    if stream is not None:
        _hold(stream, st)
    gdn_kv_append(cache.desc, p, k, v, block_table, ctx_lens, cu_seqlens, st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "kv_append (device status)")


def gdn_kv_read(cache, p, block_table, start, cu_seqlens, k_out, v_out, dev_status=None,
                stream=None):
    _check(_lib.gdn_kv_read(cache, p, block_table.data_ptr(), _opt(start), _opt(cu_seqlens),
                            k_out.data_ptr(), v_out.data_ptr(), _opt(dev_status),
                            _stream(stream)), "gdn_kv_read")


def kv_read(cache, block_table, start, cu_seqlens, tokens, dtype=torch.bfloat16,
            check_status=False, stream=None):
    """Keys and values [tokens, hkv, D] of the positions start[n] onward (None: from 0) of each
    sequence, cu_seqlens[n + 1] - cu_seqlens[n] of them, read back from the cache."""
    where = "kv_read"
    io = _IO.get(dtype)
    if io is None:
        _refuse(where, f"dtype {dtype}", _GDN_ERR_UNSUPPORTED)
    N, max_pages = _kv_sequences(where, tokens, block_table, start, cu_seqlens)
    shape, device = (tokens, cache.heads, cache.head_dim), block_table.device
    k = torch.empty(shape, dtype=dtype, device=device)
    v = torch.empty(shape, dtype=dtype, device=device)
    p = KvProblem(tokens, N, max_pages, 0, io, 0, 0, 0, 0, 0, 0)
    st = torch.zeros(1, dtype=_I32, device=device) if check_status else None
    if stream is not None:
        _hold(stream, k, v, st)
    gdn_kv_read(cache.desc, p, block_table, start, cu_seqlens, k, v, st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "kv_read (device status)")
    return k, v


def gdn_kv_attention_workspace_size(cache, p) -> int:
    return _lib.gdn_kv_attention_workspace_size(cache, p)


def gdn_kv_attention(cache, p, q, block_table, kv_lens, cu_seqlens, scale, window, out, lse,
                     workspace, ws_bytes=None, dev_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_kv_attention(cache, p, q.data_ptr(), block_table.data_ptr(),
                                 kv_lens.data_ptr(), _opt(cu_seqlens), scale, window,
                                 out.data_ptr(), _opt(lse), workspace.data_ptr(), ws_bytes,
                                 _opt(dev_status), _stream(stream)), "gdn_kv_attention")


def kv_attention(cache, q, block_table, kv_lens, cu_seqlens=None, scale=None, window=0,
                 workspace=None, check_status=False, stream=None):
    """out [T, hq, D] and lse [T, hq] of the queries of each sequence's last tokens over the
    cache's kv_lens[n] tokens (which include them); scale defaults to 1 / sqrt(D).  Without
    cu_seqlens the rows are one sequence's, or one row each of T sequences."""
    where = "kv_attention"
    io, dtype, device = _io_of(where, q), q.dtype, q.device
    shape, qt, qh = _rows(where, "q", q, dtype)
    T, hq, D = shape
    if D != cache.head_dim:
        _refuse(where, f"q {tuple(shape)} for a cache of heads of {cache.head_dim}")
    N, max_pages = _kv_sequences(where, T, block_table, kv_lens, cu_seqlens)
    p = KvProblem(T, N, max_pages, hq, io, 0, 0, 0, 0, qt, qh)
    out = torch.empty(shape, dtype=dtype, device=device)
    lse = torch.empty((T, hq), dtype=_F32, device=device)
    if workspace is None:
        workspace = torch.empty(gdn_kv_attention_workspace_size(cache.desc, p),
                                dtype=torch.uint8, device=device)
    st = torch.zeros(1, dtype=_I32, device=device) if check_status else None
    if stream is not None:
        _hold(stream, out, lse, workspace, st)
    gdn_kv_attention(cache.desc, p, q, block_table, kv_lens, cu_seqlens,
                     D ** -0.5 if scale is None else scale, window, out, lse, workspace, None,
                     st, stream)
    if check_status:
        _check(gdn_device_status(st, True, stream), "kv_attention (device status)")
    return out, lse


# ------------------------------------------------------------------ convenience API

def workspace_for(p: Problem, device="cuda") -> torch.Tensor:
    return torch.empty(max(gdn_workspace_size(p), 256), dtype=torch.uint8, device=device)


def forward(q, k, v, g, beta, h0=None, cu_seqlens=None, P=1, out=None,
            h_final=None, workspace=None, want_final=True, check_status=False, stream=None):
    """out, h_final = forward(...) on CUDA tensors (layouts of include/gdn.h).

    ``cu_seqlens`` is an int32 CUDA tensor [N+1] or None (one sequence).  With
    ``check_status`` the device status word is read back (a synchronisation)."""
    p = problem_for(q, v, cu_seqlens, P)
    N = p.num_seqs
    if out is None:
        out = torch.empty_like(v)
    if h_final is None and want_final:
        h_final = torch.empty(N, p.hv, p.k_dim, p.v_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(p, q.device)
    gdn_forward(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace, stream=stream)
    if check_status:
        st = gdn_device_status(workspace, True, stream)
        _check(st, "gdn_forward (device status)")
    return out, h_final
