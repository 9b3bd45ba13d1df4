"""ctypes binding of libgdn.so (the C ABI declared in include/gdn.h).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  Functions named after the C entry points take torch CUDA tensors, pass their
data pointers and the current torch stream, and raise ``GdnError`` on a non-OK status.
``forward()`` is the convenience call that allocates the outputs and the workspace.

Importing this module loads the library and raises ImportError when it has not been built
(``python -m gated_delta_rule_07_gb300.build``).  The softmax-attention layers' calls also need
the torch binding beside it, which their first use loads, with the same ImportError; the recurrent
calls do without.  There is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build

LIB_PATH = _build.LIB

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libgdn.so is not built ({LIB_PATH}); run "
                      "`python -m gated_delta_rule_07_gb300.build` (needs nvcc)")

# (global: the torch binding's references to the C entry points are resolved against it)
_lib = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_GLOBAL)


def _load_torch_binding():
    path = _build.TORCH_LIB
    if not os.path.exists(path):
        raise ImportError(f"_gdn_torch.so is not built ({path}); run "
                          "`python -m gated_delta_rule_07_gb300.build`")
    loader = importlib.machinery.ExtensionFileLoader("_gdn_torch", path)
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gdn_torch", loader))
    loader.exec_module(mod)
    return mod


class _Unloaded:
    """Stands for the torch binding until a call of it is looked up."""

    def __getattr__(self, name):
        global _native
        _native = _load_torch_binding()
        _native.set_error(GdnError)
        return getattr(_native, name)


_native = _Unloaded()

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
            "gdn_kv_attention", "gdn_check_linear_problem", "gdn_linear_attention_workspace_size",
            "gdn_linear_attention", "gdn_linear_attention_backward_workspace_size",
            "gdn_linear_attention_backward", "gdn_linear_attention_decode", "gdn_checkpoint_pack",
            "gdn_checkpoint_open")


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


class LinearProblem(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("hk", ctypes.c_int32), ("hv", ctypes.c_int32), ("k_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64)]


class LinearSaved(ctypes.Structure):
    _fields_ = [("q_codes", ctypes.c_void_p), ("k_codes", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("format", ctypes.c_int32)]


class CheckpointDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("total_tokens", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


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
_lp = ctypes.POINTER(LinearProblem)
_lib.gdn_check_linear_problem.argtypes = [_lp]
_lib.gdn_linear_attention_workspace_size.restype = ctypes.c_size_t
_lib.gdn_linear_attention_workspace_size.argtypes = [_lp]
_lib.gdn_linear_attention.argtypes = [_lp, _vp, _vp, _vp, _fp, _fp, _ip, _vp, _fp, _vp,
                                      ctypes.c_size_t, _ip, _vp]
_lib.gdn_linear_attention_backward_workspace_size.restype = ctypes.c_size_t
_lib.gdn_linear_attention_backward_workspace_size.argtypes = [_lp, ctypes.c_int]
_lib.gdn_linear_attention_backward.argtypes = [_lp, _vp, _vp, _vp, ctypes.POINTER(LinearSaved), _fp,
                                               _fp, _ip, _vp, _fp, _vp, _vp, _vp, _fp, _vp,
                                               ctypes.c_size_t, _ip, _vp]
_lib.gdn_linear_attention_decode.argtypes = [_lp, ctypes.c_int32, _vp, _vp, _vp, _fp, _ip, _fp, _vp,
                                             _ip, _vp]
_lib.gdn_checkpoint_pack.argtypes = [ctypes.POINTER(CheckpointDesc), ctypes.c_int32, ctypes.c_int32,
                                     _ip, _vp]
_lib.gdn_checkpoint_open.argtypes = [ctypes.POINTER(CheckpointDesc), ctypes.c_int32, ctypes.c_int32,
                                     _vp]
for _n in EXPORTED:
    if _n not in ("gdn_status_string", "gdn_workspace_size", "gdn_last_error_string",
                  "gdn_backward_workspace_size", "gdn_qk_norm_rope_backward_workspace_size",
                  "gdn_kv_attention_workspace_size", "gdn_linear_attention_workspace_size",
                  "gdn_linear_attention_backward_workspace_size"):
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


def _side_stream(stream, inputs):
    """A torch stream for what a call was given (one of torch's, or an integer handle), on the GPU of
    the call's tensors."""
    gpu = next((t.device for t in inputs if getattr(t, "is_cuda", False)), None)
    if not hasattr(stream, "cuda_stream"):
        # (0 and 1 are CUDA's names of the legacy default stream)
        return torch.cuda.default_stream(gpu) if int(stream) in (0, 1) else (
            torch.cuda.ExternalStream(int(stream), device=gpu))
    if gpu is not None and stream.device != gpu:
        raise GdnError(1, f"the stream is on {stream.device}, the tensors on {gpu}")
    return stream


def _on(stream, call, *inputs):
    """call() with `stream` as torch's current one, so that everything it allocates, clears and
    launches is ordered on it.  The allocator learns that the inputs are used there and that the
    outputs will be used on the caller's stream: no memory is handed out again before the work that
    uses it is done.  Ordering the streams themselves (inputs written, outputs read) is the caller's."""
    side = _side_stream(stream, inputs)
    with torch.cuda.stream(side):
        result = call()
    here = torch.cuda.current_stream(side.device)
    if here != side:
        for t in inputs:
            if isinstance(t, torch.Tensor):
                t.record_stream(side)
        for t in result if isinstance(result, tuple) else (result,):
            if t is not None:
                t.record_stream(here)
    return result


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
    forward on the same inputs; allocates the outputs (and the workspace unless given).  q, k and v
    are the tensors or their Checkpoints."""
    if stream is not None:
        held = [t for x in (q, k, v) for t in
                ((x.codes, x.scale) if isinstance(x, Checkpoint) else (x,))]
        return _on(stream, lambda: backward(q, k, v, g, beta, dout, h0, dh_final, cu_seqlens,
                                            workspace, check_status),
                   *held, g, beta, dout, h0, dh_final, cu_seqlens, workspace)
    q, k, v = (checkpoint_open(x)[0] if isinstance(x, Checkpoint) else x for x in (q, k, v))
    p = problem_for(q, v, cu_seqlens)
    N = p.num_seqs
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    dh0 = torch.empty(N, p.hv, p.k_dim, p.v_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(gdn_backward_workspace_size(p), 256), dtype=torch.uint8,
                                device=q.device)
    gdn_backward(p, q, k, v, g, beta, h0, cu_seqlens, dout, dh_final, dq, dk, dv, dg, dbeta,
                 dh0, workspace)
    if check_status:
        _check(gdn_device_status(workspace), "gdn_backward (device status)")
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
    if stream is not None:
        return _on(stream, lambda: prologue(x, conv_w, a, b, A_log, dt_bias, hk, hv, K, V,
                                            conv_state, cu_seqlens, activation, check_status),
                   x, conv_w, a, b, A_log, dt_bias, conv_state, cu_seqlens)
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
                 new_state if W > 1 else None, st)
    if check_status:
        _check(gdn_device_status(st), "gdn_prologue (device status)")
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
    if stream is not None:
        return _on(stream, lambda: decode(q, k, v, g, beta, slot, state, out, check_status),
                   q, k, v, g, beta, slot, state, out)
    p = decode_problem_for(q, v, state)
    if out is None:
        out = torch.empty_like(v)
    st = torch.zeros(1, dtype=torch.int32, device=q.device) if check_status else None
    gdn_decode_step(p, q, k, v, g, beta, slot, state, out, st)
    if check_status:
        _check(gdn_device_status(st), "gdn_decode_step (device status)")
    return out


def gdn_device_status(status_word, reset=True, stream=None) -> int:
    """Synchronous read of a device status word (a dev_status tensor or a workspace)."""
    return _lib.gdn_device_status(_ptr(status_word), int(bool(reset)), _stream(stream))


# ------------------------------------------------- softmax-attention layers' operators
#
# The functions named after the C entry points are the ctypes form, as above.  The others go
# through the torch binding (csrc/gdn_torch.cpp): a decode step's kernels take a few microseconds,
# so its checks and allocations are made there.  What they refuse raises GdnError before any CUDA
# work.

_IO = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_KV_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}
_ROPE_STYLES = {"half": 0, "pairs": 1}


def _refuse(where, why, status=1):
    raise GdnError(status, f"{where}: {why}")


def _checked(check_status, device, where, call):
    """call(status word or None), with the word read back afterwards where asked for."""
    if not check_status:
        return call(None)
    st = torch.zeros(1, dtype=torch.int32, device=device)
    result = call(st)
    _check(gdn_device_status(st), f"{where} (device status)")
    return result


def gdn_qk_norm_rope(p, q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out,
                     dev_status=None, stream=None):
    _check(_lib.gdn_qk_norm_rope(p, _ptr(q), _ptr(k), _ptr(positions), _ptr(cos_sin),
                                 _ptr(q_weight), _ptr(k_weight), _ptr(q_out), _ptr(k_out),
                                 _ptr(dev_status), _stream(stream)), "gdn_qk_norm_rope")


def qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, style="half", check_status=False, stream=None):
    """Queries [T, hq, D] and keys [T, hkv, D], normalised per head and rotated by position (see
    include/gdn.h); q and k may be slices of one projection.  Returns contiguous tensors."""
    if stream is not None:
        return _on(stream, lambda: qk_norm_rope(q, k, positions, cos_sin, q_weight, k_weight, eps,
                                                weight_offset, style, check_status),
                   q, k, positions, cos_sin, q_weight, k_weight)
    code = _ROPE_STYLES.get(style)
    if code is None:
        _refuse("qk_norm_rope", f"style {style!r}")
    if not check_status:
        return _native.qk_norm_rope(q, k, positions, cos_sin, q_weight, k_weight, eps,
                                    weight_offset, code, None)
    return _checked(True, q.device, "qk_norm_rope", lambda st: _native.qk_norm_rope(
        q, k, positions, cos_sin, q_weight, k_weight, eps, weight_offset, code, st))


def gdn_qk_norm_rope_backward_workspace_size(p) -> int:
    return _lib.gdn_qk_norm_rope_backward_workspace_size(p)


def gdn_qk_norm_rope_backward(p, q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out,
                              dq, dk, dq_weight, dk_weight, workspace, ws_bytes=None,
                              dev_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_qk_norm_rope_backward(
        p, _ptr(q), _ptr(k), _ptr(positions), _ptr(cos_sin), _ptr(q_weight), _ptr(k_weight),
        _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dq_weight), _ptr(dk_weight),
        _ptr(workspace), int(ws_bytes), _ptr(dev_status), _stream(stream)),
        "gdn_qk_norm_rope_backward")


def qk_norm_rope_backward(q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out, eps=1e-6,
                          weight_offset=0.0, style="half", workspace=None, check_status=False,
                          stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of <dq_out, q_out> + <dk_out, k_out> through
    qk_norm_rope on the same inputs."""
    where = "qk_norm_rope_backward"
    if stream is not None:
        return _on(stream, lambda: qk_norm_rope_backward(
            q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out, eps, weight_offset, style,
            workspace, check_status), q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out,
            workspace)
    code = _ROPE_STYLES.get(style)
    if code is None:
        _refuse(where, f"style {style!r}")
    if not check_status:
        return _native.qk_norm_rope_backward(q, k, positions, cos_sin, q_weight, k_weight, dq_out,
                                             dk_out, eps, weight_offset, code, workspace, None)
    return _checked(True, q.device, where, lambda st: _native.qk_norm_rope_backward(
        q, k, positions, cos_sin, q_weight, k_weight, dq_out, dk_out, eps, weight_offset, code,
        workspace, st))


class _CacheHandle(ctypes.Structure):
    """What the torch binding reads of a cache: its description and the GPU that it is on."""
    _fields_ = [("desc", KvCacheDesc), ("device", ctypes.c_int32)]


class KVCache:
    """The buffers of a paged 8-bit key/value cache (layouts of include/gdn.h):
    k [pages, hkv, page, D] and v [pages, hkv, page // 4, D, 4], both int8 or float8_e4m3fn;
    k_scale, v_scale [pages, hkv] fp32.  ``KVCache.empty`` allocates them.  The buffers of a cache
    stay the ones that it was made of (its calls keep their addresses); their contents are free."""

    def __init__(self, k, v, k_scale, v_scale):
        fmt = _KV_FORMATS.get(k.dtype)
        if fmt is None:
            _refuse("KVCache", f"dtype {k.dtype}", 2)
        if k.dim() != 4:
            _refuse("KVCache", "k is to be [pages, hkv, page, D]")
        pages, hkv, page, D = k.shape
        for name, t, shape, dtype in (("k", k, k.shape, k.dtype),
                                      ("v", v, (pages, hkv, page // 4, D, 4), k.dtype),
                                      ("k_scale", k_scale, (pages, hkv), torch.float32),
                                      ("v_scale", v_scale, (pages, hkv), torch.float32)):
            if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda:
                _refuse("KVCache", f"{name} is to be a contiguous {dtype} tensor {tuple(shape)} on "
                                   f"the GPU, got {t.dtype} {tuple(t.shape)} on {t.device}")
            if t.device != k.device:
                _refuse("KVCache", f"{name} is on {t.device}, k on {k.device}")
        self._buffers = k, v, k_scale, v_scale
        self._handle = _CacheHandle(KvCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                                v_scale.data_ptr(), pages, page, hkv, D, fmt),
                                    k.device.index)
        self.desc = self._handle.desc  # (a view of it)
        self._address = ctypes.addressof(self._handle)

    buffers = property(lambda self: self._buffers)
    k = property(lambda self: self._buffers[0])
    v = property(lambda self: self._buffers[1])
    k_scale = property(lambda self: self._buffers[2])
    v_scale = property(lambda self: self._buffers[3])

    @classmethod
    def empty(cls, pages, hkv, page, D, dtype=torch.int8, device="cuda"):
        """A cache of `pages` pages; nothing in it is initialised, or needs to be."""
        return cls(torch.empty(pages, hkv, page, D, dtype=dtype, device=device),
                   torch.empty(pages, hkv, page // 4, D, 4, dtype=dtype, device=device),
                   torch.empty(pages, hkv, dtype=torch.float32, device=device),
                   torch.empty(pages, hkv, dtype=torch.float32, device=device))


def gdn_kv_append(cache, p, k, v, block_table, ctx_lens, cu_seqlens, dev_status=None,
                  stream=None):
    _check(_lib.gdn_kv_append(cache, p, _ptr(k), _ptr(v), _ptr(block_table), _ptr(ctx_lens),
                              _ptr(cu_seqlens), _ptr(dev_status), _stream(stream)),
           "gdn_kv_append")


def kv_append(cache, k, v, block_table, ctx_lens, cu_seqlens=None, check_status=False,
              stream=None):
    """Quantises new keys and values [T, hkv, D] into the cache's pages, behind the ctx_lens[n]
    tokens that each sequence already holds.  Without cu_seqlens the rows are one sequence's, or
    one row each of T sequences."""
    if stream is not None:
        return _on(stream, lambda: kv_append(cache, k, v, block_table, ctx_lens, cu_seqlens,
                                             check_status),
                   k, v, block_table, ctx_lens, cu_seqlens, *cache.buffers)
    if not check_status:
        _native.kv_append(cache._address, k, v, block_table, ctx_lens, cu_seqlens, None)
        return
    _checked(True, k.device, "kv_append", lambda st: _native.kv_append(
        cache._address, k, v, block_table, ctx_lens, cu_seqlens, st))


def gdn_kv_read(cache, p, block_table, start, cu_seqlens, k_out, v_out, dev_status=None,
                stream=None):
    _check(_lib.gdn_kv_read(cache, p, _ptr(block_table), _ptr(start), _ptr(cu_seqlens),
                            _ptr(k_out), _ptr(v_out), _ptr(dev_status), _stream(stream)),
           "gdn_kv_read")


def kv_read(cache, block_table, start, cu_seqlens, tokens, dtype=torch.bfloat16,
            check_status=False, stream=None):
    """Keys and values [tokens, hkv, D] of the positions start[n] onward (None: from 0) of each
    sequence, cu_seqlens[n + 1] - cu_seqlens[n] of them, read back from the cache."""
    if stream is not None:
        return _on(stream, lambda: kv_read(cache, block_table, start, cu_seqlens, tokens, dtype,
                                           check_status),
                   block_table, start, cu_seqlens, *cache.buffers)
    io = _IO.get(dtype)
    if io is None:
        _refuse("kv_read", f"dtype {dtype}", 2)
    if not check_status:
        return _native.kv_read(cache._address, block_table, start, cu_seqlens, tokens, io, None)
    return _checked(True, block_table.device, "kv_read", lambda st: _native.kv_read(
        cache._address, block_table, start, cu_seqlens, tokens, io, st))


def gdn_kv_attention_workspace_size(cache, p) -> int:
    return _lib.gdn_kv_attention_workspace_size(cache, p)


def gdn_kv_attention(cache, p, q, block_table, kv_lens, cu_seqlens, scale, window, out, lse,
                     workspace, ws_bytes=None, dev_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_kv_attention(cache, p, _ptr(q), _ptr(block_table), _ptr(kv_lens),
                                 _ptr(cu_seqlens), scale, window, _ptr(out), _ptr(lse),
                                 _ptr(workspace), int(ws_bytes), _ptr(dev_status),
                                 _stream(stream)), "gdn_kv_attention")


def kv_attention_workspace(cache, q, block_table):
    """A workspace for kv_attention calls of these shapes."""
    if q.dim() != 3 or block_table.dim() != 2:
        _refuse("kv_attention_workspace", "q is to be [tokens, heads, D], block_table [N, pages]")
    if q.dtype not in _IO:
        _refuse("kv_attention_workspace", f"dtype {q.dtype}", 2)
    T, hq, _ = q.shape
    p = KvProblem(T, block_table.shape[0], block_table.shape[1], hq, _IO[q.dtype], 0, 0, 0, 0,
                  q.stride(0), q.stride(1))
    return torch.empty(gdn_kv_attention_workspace_size(cache.desc, p), dtype=torch.uint8,
                       device=q.device)


def kv_attention(cache, q, block_table, kv_lens, cu_seqlens=None, scale=None, window=0,
                 workspace=None, check_status=False, stream=None):
    """out [T, hq, D] and lse [T, hq] of the queries of each sequence's last tokens over the
    cache's kv_lens[n] tokens (which include them); scale defaults to 1 / sqrt(D).  Without
    cu_seqlens the rows are one sequence's, or one row each of T sequences."""
    if stream is not None:
        return _on(stream, lambda: kv_attention(cache, q, block_table, kv_lens, cu_seqlens, scale,
                                                window, workspace, check_status),
                   q, block_table, kv_lens, cu_seqlens, workspace, *cache.buffers)
    if not check_status:
        return _native.kv_attention(cache._address, q, block_table, kv_lens, cu_seqlens, scale,
                                    window, workspace, None)
    return _checked(True, q.device, "kv_attention", lambda st: _native.kv_attention(
        cache._address, q, block_table, kv_lens, cu_seqlens, scale, window, workspace, st))


# ------------------------------------------------- linear attention with a decay for each head

def gdn_check_linear_problem(p) -> int:
    return _lib.gdn_check_linear_problem(p)


def gdn_linear_attention_workspace_size(p) -> int:
    return _lib.gdn_linear_attention_workspace_size(p)


def gdn_linear_attention(p, q, k, v, log_decay, h0, cu_seqlens, out, h_final, workspace,
                         ws_bytes=None, dev_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_linear_attention(p, _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(h0),
                                     _ptr(cu_seqlens), _ptr(out), _ptr(h_final), _ptr(workspace),
                                     int(ws_bytes), _ptr(dev_status), _stream(stream)),
           "gdn_linear_attention")


def linear_attention(q, k, v, log_decay, h0=None, cu_seqlens=None, workspace=None,
                     check_status=False, stream=None):
    """out [T, hv, V] and the final states [N, hv, K, V] of h_t = exp(log_decay) h_{t-1} + k_t v_t^T,
    out_t = h_t^T q_t over packed sequences (see include/gdn.h): q, k [T, hk, K] and v [T, hv, V]
    may be slices of one projection, log_decay [hv] <= 0 belongs to the layer.  bf16 tensors go through
    fp16 operands, float32 ones (.float() of them too) are computed in fp32 throughout."""
    if stream is not None:
        return _on(stream, lambda: linear_attention(q, k, v, log_decay, h0, cu_seqlens, workspace,
                                                    check_status),
                   q, k, v, log_decay, h0, cu_seqlens, workspace)
    if not check_status:
        return _native.linear_attention(q, k, v, log_decay, h0, cu_seqlens, workspace, None)
    return _checked(True, q.device, "linear_attention", lambda st: _native.linear_attention(
        q, k, v, log_decay, h0, cu_seqlens, workspace, st))


def gdn_linear_attention_backward_workspace_size(p, saved=False) -> int:
    return _lib.gdn_linear_attention_backward_workspace_size(p, int(bool(saved)))


def gdn_linear_attention_backward(p, q, k, v, saved, log_decay, h0, cu_seqlens, dout, dh_final, dq,
                                  dk, dv, dh0, workspace, ws_bytes=None, dev_status=None,
                                  stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if ws_bytes is None else ws_bytes
    _check(_lib.gdn_linear_attention_backward(
        p, _ptr(q), _ptr(k), _ptr(v), saved, _ptr(log_decay), _ptr(h0), _ptr(cu_seqlens),
        _ptr(dout), _ptr(dh_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dh0), _ptr(workspace),
        int(ws_bytes), _ptr(dev_status), _stream(stream)), "gdn_linear_attention_backward")


def linear_attention_backward(q, k, v, log_decay, dout, h0=None, dh_final=None, cu_seqlens=None,
                              workspace=None, check_status=False, stream=None):
    """Gradients (dq, dk, dv, dh0) of <dout, out> + <dh_final, h_final> through linear_attention on
    the same inputs.  q, k and v are the tensors, or all three their Checkpoints."""
    where = "linear_attention_backward"
    held = [isinstance(x, Checkpoint) for x in (q, k, v)]
    if any(held) and not all(held):
        _refuse(where, "q, k and v are to be tensors, or all of them checkpoints")
    if all(held):
        if not q.dtype == k.dtype == v.dtype:
            _refuse(where, "the checkpoints' dtypes differ")
        acts = (q.codes, k.codes, v.codes, q.scale, k.scale, v.scale, _IO[q.dtype])
    else:
        acts = (q, k, v, None, None, None, None)
    if stream is not None:
        return _on(stream, lambda: linear_attention_backward(q, k, v, log_decay, dout, h0, dh_final,
                                                             cu_seqlens, workspace, check_status),
                   *acts[:6], log_decay, dout, h0, dh_final, cu_seqlens, workspace)
    if not check_status:
        return _native.linear_attention_backward(*acts, log_decay, dout, h0, dh_final, cu_seqlens,
                                                 workspace, None)
    return _checked(True, dout.device, where, lambda st: _native.linear_attention_backward(
        *acts, log_decay, dout, h0, dh_final, cu_seqlens, workspace, st))


def gdn_linear_attention_decode(p, slots, q, k, v, log_decay, slot, state, out, dev_status=None,
                                stream=None):
    _check(_lib.gdn_linear_attention_decode(p, int(slots), _ptr(q), _ptr(k), _ptr(v),
                                            _ptr(log_decay), _ptr(slot), _ptr(state), _ptr(out),
                                            _ptr(dev_status), _stream(stream)),
           "gdn_linear_attention_decode")


def linear_attention_decode(q, k, v, log_decay, slot, state, check_status=False, stream=None):
    """One token of each request: row b continues the request held in state[slot[b]] (updated in
    place; state [slots, hv, K, V] fp32, slot int32 [B], negative for padding rows).  Returns
    out [B, hv, V]."""
    if stream is not None:
        return _on(stream, lambda: linear_attention_decode(q, k, v, log_decay, slot, state,
                                                           check_status),
                   q, k, v, log_decay, slot, state)
    if not check_status:
        return _native.linear_attention_decode(q, k, v, log_decay, slot, state, None)[0]
    return _checked(True, q.device, "linear_attention_decode",
                    lambda st: _native.linear_attention_decode(q, k, v, log_decay, slot, state,
                                                               st))[0]


# ------------------------------------------------- activations held in 8 bits

class Checkpoint:
    """Rows [T, heads, D] held in 8 bits (layouts of include/gdn.h): codes [T, heads, D] int8 or
    float8_e4m3fn, scale [T, heads] fp32, and the dtype that they open to.  checkpoint_pack makes
    them."""

    __slots__ = ("codes", "scale", "dtype")

    def __init__(self, codes, scale, dtype=torch.bfloat16):
        if codes.dtype not in _KV_FORMATS or dtype not in _IO:
            _refuse("Checkpoint", f"codes of dtype {codes.dtype} for {dtype}", 2)
        for name, t, shape in (("codes", codes, codes.shape), ("scale", scale, codes.shape[:2])):
            if codes.dim() != 3 or t.shape != shape or not t.is_contiguous() or not t.is_cuda or \
                    t.device != codes.device or (t is scale and t.dtype is not torch.float32):
                _refuse("Checkpoint", f"{name} of {t.dtype} {tuple(t.shape)} on {t.device}")
        self.codes, self.scale, self.dtype = codes, scale, dtype

    shape = property(lambda self: self.codes.shape)

    def __repr__(self):
        return f"Checkpoint({tuple(self.shape)}, {self.codes.dtype} for {self.dtype})"


def gdn_checkpoint_pack(tensors, count, format, dev_status=None, stream=None):
    _check(_lib.gdn_checkpoint_pack(tensors, int(count), int(format), _ptr(dev_status),
                                    _stream(stream)), "gdn_checkpoint_pack")


def checkpoint_pack(*tensors, dtype=torch.int8, check_status=False, stream=None):
    """Checkpoints of up to 8 tensors [T, heads, D] (slices of one projection are fine), one scale for
    each row of D elements, int8 or float8_e4m3fn.  With check_status, raises where a value was not
    finite."""
    if stream is not None:
        made = _on(stream, lambda: tuple(x for c in checkpoint_pack(
            *tensors, dtype=dtype, check_status=check_status) for x in (c.codes, c.scale)), *tensors)
    else:
        fmt = _KV_FORMATS.get(dtype)
        if fmt is None:
            _refuse("checkpoint_pack", f"dtype {dtype}", 2)
        if not tensors:
            _refuse("checkpoint_pack", "nothing to hold")
        if not check_status:
            made = _native.checkpoint_pack(None, fmt, *tensors)
        else:
            made = _checked(True, tensors[0].device, "checkpoint_pack",
                            lambda st: _native.checkpoint_pack(st, fmt, *tensors))
    parts = iter(made)
    return tuple([_checkpoint(codes, scale, x.dtype) for x, codes, scale in zip(tensors, parts, parts)])


def _checkpoint(codes, scale, dtype):
    c = Checkpoint.__new__(Checkpoint)  # (what the library has made needs no checks)
    c.codes, c.scale, c.dtype = codes, scale, dtype
    return c


def gdn_checkpoint_open(tensors, count, format, stream=None):
    _check(_lib.gdn_checkpoint_open(tensors, int(count), int(format), _stream(stream)),
           "gdn_checkpoint_open")


def checkpoint_open(*checkpoints, stream=None):
    """The tensors that checkpoints stand for, contiguous and in their dtypes."""
    if stream is not None:
        return _on(stream, lambda: checkpoint_open(*checkpoints),
                   *(t for c in checkpoints for t in (c.codes, c.scale)))
    if not checkpoints:
        _refuse("checkpoint_open", "nothing to open")
    return _native.checkpoint_open(*[x for c in checkpoints
                                     for x in (c.codes, c.scale, _IO[c.dtype])])


# ------------------------------------------------------------------ convenience API

def workspace_for(p: Problem, device="cuda") -> torch.Tensor:
    return torch.empty(max(gdn_workspace_size(p), 256), dtype=torch.uint8, device=device)


def forward(q, k, v, g, beta, h0=None, cu_seqlens=None, P=1, out=None,
            h_final=None, workspace=None, want_final=True, check_status=False, stream=None):
    """out, h_final = forward(...) on CUDA tensors (layouts of include/gdn.h).

    ``cu_seqlens`` is an int32 CUDA tensor [N+1] or None (one sequence).  With
    ``check_status`` the device status word is read back (a synchronisation)."""
    if stream is not None:
        return _on(stream, lambda: forward(q, k, v, g, beta, h0, cu_seqlens, P, out, h_final,
                                           workspace, want_final, check_status),
                   q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace)
    p = problem_for(q, v, cu_seqlens, P)
    N = p.num_seqs
    if out is None:
        out = torch.empty_like(v)
    if h_final is None and want_final:
        h_final = torch.empty(N, p.hv, p.k_dim, p.v_dim, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(p, q.device)
    gdn_forward(p, q, k, v, g, beta, h0, cu_seqlens, out, h_final, workspace)
    if check_status:
        st = gdn_device_status(workspace)
        _check(st, "gdn_forward (device status)")
    return out, h_final
