"""KDA (Kimi Delta Attention) gated delta-rule recurrence on B200 (sm_100a).

Thin Python binding of ``libkda.so`` (C ABI in ``include/kda.h``).  This module
only marshals arguments: it checks shapes, allocates outputs and the workspace
with torch (device memory and streams are all torch is used for) and calls the
library.  Every step of the computation runs in the library's CUDA kernels;
there is no CPU or PyTorch fallback.  If the library is missing or no CUDA
device is present the calls raise.

Entry points (same names as the C ABI):
  chunk_fwd      chunkwise prefill: (o or y, final_state)
  decode_step    one recurrent step per sequence, state updated in place
  gate_norm      per-head RMSNorm over dv times sigmoid output gate
  workspace_size bytes the prefill needs
  chunk_bwd      gradients of the prefill (without the gate)
  kcp_transition / kcp_compose / kcp_finish
                 the per-device steps of context parallelism across devices
                 (the exchange between them is in ``kcp.py``)
  scan_fwd / scan_bwd / scan_decode_step(s)
                 the element-wise gated scan: prefill, gradients, single tokens
  gate_norm_bwd  gradients of gate_norm
  state_copy / state_alloc / state_free / state_compact
                 pages of recurrent states in a pool: copy, fork, clear, take, free
                 and compact (decode_step(s) and scan_decode_step(s) take `slots`)
  query_status   reads and clears the device status word of a workspace
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK = 0
KDA_F32, KDA_BF16 = 0, 1
HEAD_DIM = 128
SCAN_CHUNK = 8  # tokens between two rows of scan_fwd's chunk_states
COPY_LIST = 65535  # page moves that one kda_state_copy takes

_STATUS_NAMES = {
    0: "KDA_OK", -1: "KDA_ERR_INVALID_ARG", -2: "KDA_ERR_UNSUPPORTED", -3: "KDA_ERR_MISALIGNED",
    -4: "KDA_ERR_WORKSPACE", -5: "KDA_ERR_CUDA", -6: "KDA_ERR_TIMEOUT", -7: "KDA_ERR_DEVICE_ARG",
}


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 16), ("launches", ctypes.c_int), ("ms", ctypes.c_double)]


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS_NAMES.get(status, status)} ({status})")


_lib = None


def load_library(path: str | None = None):
    """Loads libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with `python -m linear_attention_recurrence_06_b200.build` "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [i32]
    lib.kda_version.restype = i32
    lib.kda_chunk_fwd_workspace_size.restype = i32
    lib.kda_chunk_fwd_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.kda_chunk_fwd.restype = i32
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, i32, i64,
                                  i32, i32, f32, vp, vp, f32, vp, sz, vp]
    lib.kda_chunk_fwd_ckpt.restype = i32
    lib.kda_chunk_fwd_ckpt.argtypes = list(lib.kda_chunk_fwd.argtypes[:22]) + [vp, i64] + \
        list(lib.kda_chunk_fwd.argtypes[22:])
    lib.kda_chunk_fwd_segmented.restype = i32
    lib.kda_chunk_fwd_segmented.argtypes = list(lib.kda_chunk_fwd.argtypes[:22]) + [i32] + \
        list(lib.kda_chunk_fwd.argtypes[22:])
    lib.kda_chunk_fwd_segmented_workspace_size.restype = i32
    lib.kda_chunk_fwd_segmented_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64, i32, ctypes.POINTER(sz)]
    lib.kda_kcp_workspace_size.restype = i32
    lib.kda_kcp_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64, ctypes.POINTER(sz)]
    lib.kda_kcp_transition.restype = i32
    lib.kda_kcp_transition.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, i32, i64, i32, f32, vp, vp,
                                       sz, vp]
    lib.kda_kcp_compose.restype = i32
    lib.kda_kcp_compose.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp]
    lib.kda_kcp_finish.restype = i32
    lib.kda_kcp_finish.argtypes = [vp, vp, vp, i32, i64, i32, i32, i32, vp, i32, i64, i32, i32, vp, vp, f32, vp, sz,
                                   vp]
    lib.kda_chunk_bwd_workspace_size.restype = i32
    lib.kda_chunk_bwd_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64, ctypes.POINTER(sz)]
    lib.kda_chunk_bwd.restype = i32
    lib.kda_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                  vp, i32, i64, i32, f32, vp, sz, vp]
    lib.kda_decode_step.restype = i32
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, f32, vp]
    lib.kda_decode_steps.restype = i32
    lib.kda_decode_steps.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, vp, vp, f32,
                                     vp, vp]
    lib.kda_gate_norm.restype = i32
    lib.kda_gate_norm.argtypes = [vp, vp, vp, f32, vp, i64, i32, i32, i32, vp]
    ld = [i64] * 3
    lib.kda_scan_fwd.restype = i32
    lib.kda_scan_fwd.argtypes = [vp] * 7 + [i32, i64, i32] + ld + [vp, i32, i32, i32, i32, vp, sz, vp]
    lib.kda_scan_bwd.restype = i32
    lib.kda_scan_bwd.argtypes = [vp] * 11 + [i32, i64, i32] + ld + [i64, vp, i32, i32, i32, i32, vp, sz, vp]
    lib.kda_scan_bwd_workspace_size.restype = i32
    lib.kda_scan_bwd_workspace_size.argtypes = [i32, i64, i32, ctypes.POINTER(sz)]
    lib.kda_scan_decode_steps.restype = i32
    lib.kda_scan_decode_steps.argtypes = [vp] * 6 + [i32] * 7 + [vp, vp]
    lib.kda_decode_steps_paged.restype = i32
    lib.kda_decode_steps_paged.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp] + [i32] * 7 + [f32, vp, vp, f32, vp, vp]
    lib.kda_gate_norm_bwd.restype = i32
    lib.kda_gate_norm_bwd.argtypes = [vp, vp, vp, vp, f32, vp, vp, vp, i64, i32, i32, i32, vp, sz, vp]
    lib.kda_gate_norm_bwd_workspace_size.restype = i32
    lib.kda_gate_norm_bwd_workspace_size.argtypes = [i64, i32, ctypes.POINTER(sz)]
    lib.kda_state_copy.restype = i32
    lib.kda_state_copy.argtypes = [vp, vp, i32, i64, i32, i32, i64, i64, vp, vp, i32, vp]
    lib.kda_state_alloc.restype = i32
    lib.kda_state_alloc.argtypes = [vp, i32, vp, i32, vp]
    lib.kda_state_free.restype = i32
    lib.kda_state_free.argtypes = [vp, i32, vp, i32, vp]
    lib.kda_state_compact.restype = i32
    lib.kda_state_compact.argtypes = [vp, i32, vp, vp, vp, vp, vp]
    lib.kda_query_status.restype = i32
    lib.kda_query_status.argtypes = [vp, vp]
    lib.kda_chunk_fwd_noalloc.restype = i32
    lib.kda_chunk_fwd_noalloc.argtypes = list(lib.kda_chunk_fwd.argtypes[:22]) + [vp]
    lib.kda_chunk_fwd_noalloc_query_status.restype = i32
    lib.kda_chunk_fwd_noalloc_query_status.argtypes = [vp]
    lib.kda_test_drop_tile_load.restype = i32
    lib.kda_test_drop_tile_load.argtypes = [ctypes.c_ulonglong]
    lib.kda_profile_enable.restype = i32
    lib.kda_profile_enable.argtypes = [i32]
    lib.kda_profile_read.restype = i32
    lib.kda_profile_read.argtypes = [ctypes.POINTER(KernelTime), i32, ctypes.POINTER(i32)]
    if path is None:
        _lib = lib
    return lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dt(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")


def segmented_workspace_size(T: int, H: int, n_seqs: int, max_seqlen: int, segments: int, dk: int = HEAD_DIM,
                             dv: int = HEAD_DIM) -> int:
    """Workspace bytes of the segment-parallel prefill."""
    n = ctypes.c_size_t(0)
    st = load_library().kda_chunk_fwd_segmented_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, segments,
                                                               ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_segmented_workspace_size")
    return n.value


def workspace_size(T: int, H: int, n_seqs: int, max_seqlen: int, dk: int = HEAD_DIM, dv: int = HEAD_DIM):
    """(bytes_min, bytes_full) of the prefill workspace."""
    lo, hi = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = load_library().kda_chunk_fwd_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, ctypes.byref(lo), ctypes.byref(hi))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_workspace_size")
    return lo.value, hi.value


def chunk_fwd(q, k, v, log_alpha, beta, initial_state=None, *, cu_seqlens=None, max_seqlen=None,
              scale: float = 1.0, gate=None, norm_weight=None, eps: float = 1e-6, out_dtype=None,
              output_final_state: bool = True, final_state=None, out=None, workspace=None, stream=None,
              checkpoints=None, ckpt_tokens: int = 512, segments: int = 1):
    """Chunkwise KDA prefill.

    q, k, log_alpha: [B, T, H, 128]; v: [B, T, H, 128]; beta: [B, T, H] (bf16 or
    fp32, all the same dtype).  Varlen: B = 1 and cu_seqlens int32 [N+1] on the
    device plus max_seqlen (host int).  initial_state: fp32 [N, H, 128, 128] or
    None.  gate: [B, T, H, 128] or None (then o is returned unnormalised).
    Returns (o_or_y [B, T, H, 128], final_state fp32 [N, H, 128, 128] or None).
    checkpoints: None, True (allocate zeros) or fp32 [N, max_seqlen // ckpt_tokens, H, 128, 128]
    receiving the state after every ckpt_tokens tokens of each sequence (ckpt_tokens a
    multiple of 64); then the return value is (o, final_state, checkpoints).
    segments > 1: segment-parallel prefill (kda_chunk_fwd_segmented); not combined
    with checkpoints.
    """
    torch = _torch()
    _check_cuda(q, k, v, log_alpha, beta, initial_state, cu_seqlens, gate, norm_weight)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    in_dt = _dt(q)
    for t in (k, v, log_alpha, beta) + ((gate,) if gate is not None else ()):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, log_alpha, beta and gate must share one dtype")
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen (host int)")
        N = cu_seqlens.numel() - 1
    else:
        N = B
        max_seqlen = T
    odt = out_dtype if out_dtype is not None else q.dtype
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=odt, device=q.device)
    fs = final_state
    if fs is None and output_final_state:
        fs = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        if segments > 1:
            full = segmented_workspace_size(B * T if cu_seqlens is None else T, H, N, max_seqlen, segments, dk, dv)
        else:
            _, full = workspace_size(B * T if cu_seqlens is None else T, H, N, max_seqlen, dk, dv)
        workspace = torch.empty(full, dtype=torch.uint8, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state), _ptr(o), _ptr(fs),
            B, T, H, dk, dv, _ptr(cu_seqlens), N, int(max_seqlen), in_dt, _dt(o), float(scale), _ptr(gate),
            _ptr(norm_weight), float(eps))
    tail = (_ptr(workspace), workspace.numel(), _stream(stream))
    if segments > 1:
        if checkpoints is not None:
            raise ValueError("segments > 1 does not take checkpoints")
        st = load_library().kda_chunk_fwd_segmented(*args, int(segments), *tail)
        if st != KDA_OK:
            raise KdaError(st, "kda_chunk_fwd_segmented")
        return o, fs
    if checkpoints is None:
        st = load_library().kda_chunk_fwd(*args, *tail)
        if st != KDA_OK:
            raise KdaError(st, "kda_chunk_fwd")
        return o, fs
    if checkpoints is True:
        checkpoints = torch.zeros((N, int(max_seqlen) // ckpt_tokens, H, dk, dv), dtype=torch.float32,
                                  device=q.device)
    _check_cuda(checkpoints)
    st = load_library().kda_chunk_fwd_ckpt(*args, _ptr(checkpoints), int(ckpt_tokens), *tail)
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_ckpt")
    return o, fs, checkpoints


def bwd_workspace_size(T: int, H: int, n_seqs: int, max_seqlen: int, dk: int = HEAD_DIM, dv: int = HEAD_DIM) -> int:
    """Workspace bytes of chunk_bwd."""
    n = ctypes.c_size_t(0)
    st = load_library().kda_chunk_bwd_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd_workspace_size")
    return n.value


def chunk_bwd(q, k, v, log_alpha, beta, d_o, initial_state=None, d_final_state=None, *, cu_seqlens=None,
              max_seqlen=None, scale: float = 1.0, want_d_initial_state: bool = True, workspace=None, stream=None):
    """Gradients of chunk_fwd (no gate): inputs as chunk_fwd, d_o = dL/do [B, T, H, 128]
    (the inputs' dtype), d_final_state = dL/d(final state) fp32 [N, H, 128, 128] or None.
    Returns a dict of fp32 tensors: dq, dk, dv, dlog_alpha [B, T, H, 128], dbeta [B, T, H]
    and d_initial_state [N, H, 128, 128] (None when not wanted)."""
    torch = _torch()
    _check_cuda(q, k, v, log_alpha, beta, d_o, initial_state, d_final_state, cu_seqlens, workspace)
    B, T, N, maxlen = _seq_dims(q, cu_seqlens, max_seqlen)
    H, dk, dv = q.shape[2], q.shape[3], v.shape[-1]
    for t in (k, v, log_alpha, beta, d_o):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, log_alpha, beta and d_o must share one dtype")
    f32 = dict(dtype=torch.float32, device=q.device)
    g = dict(dq=torch.empty((B, T, H, dk), **f32), dk=torch.empty((B, T, H, dk), **f32),
             dv=torch.empty((B, T, H, dv), **f32), dlog_alpha=torch.empty((B, T, H, dk), **f32),
             dbeta=torch.empty((B, T, H), **f32),
             d_initial_state=torch.empty((N, H, dk, dv), **f32) if want_d_initial_state else None)
    if workspace is None:
        workspace = torch.empty(bwd_workspace_size(B * T if cu_seqlens is None else T, H, N, maxlen, dk, dv),
                                dtype=torch.uint8, device=q.device)
    st = load_library().kda_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state),
                                      _ptr(d_o), _ptr(d_final_state), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                                      _ptr(g["dlog_alpha"]), _ptr(g["dbeta"]), _ptr(g["d_initial_state"]), B, T, H,
                                      dk, dv, _ptr(cu_seqlens), N, maxlen, _dt(q), float(scale), _ptr(workspace),
                                      workspace.numel(), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd")
    return g


def _seq_dims(q, cu_seqlens, max_seqlen):
    torch = _torch()
    B, T = q.shape[0], q.shape[1]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen (host int)")
        return B, T, cu_seqlens.numel() - 1, int(max_seqlen)
    return B, T, B, T


def kcp_workspace_size(T: int, H: int, n_seqs: int, max_seqlen: int, dk: int = HEAD_DIM, dv: int = HEAD_DIM) -> int:
    """Workspace bytes shared by kcp_transition and kcp_finish."""
    n = ctypes.c_size_t(0)
    st = load_library().kda_kcp_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_kcp_workspace_size")
    return n.value


def kcp_transition(q, k, v, log_alpha, beta, *, cu_seqlens=None, max_seqlen=None, scale: float = 1.0,
                   transition=None, workspace=None, stream=None):
    """Step 1 of context parallelism across devices, for this device's token
    segment (inputs as chunk_fwd).  Returns (transition fp32 [2, N, H, 128, 128]:
    [0] = M, [1] = B with S_out = M S_in + B; workspace holding the chunk work
    for kcp_finish)."""
    torch = _torch()
    _check_cuda(q, k, v, log_alpha, beta, cu_seqlens, transition, workspace)
    B, T, N, maxlen = _seq_dims(q, cu_seqlens, max_seqlen)
    H, dk, dv = q.shape[2], q.shape[3], v.shape[-1]
    for t in (k, v, log_alpha, beta):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, log_alpha and beta must share one dtype")
    if transition is None:
        transition = torch.empty((2, N, H, dk, dk), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(kcp_workspace_size(B * T if cu_seqlens is None else T, H, N, maxlen, dk, dv),
                                dtype=torch.uint8, device=q.device)
    st = load_library().kda_kcp_transition(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), B, T, H, dk, dv,
                                           _ptr(cu_seqlens), N, maxlen, _dt(q), float(scale), _ptr(transition),
                                           _ptr(workspace), workspace.numel(), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_kcp_transition")
    return transition, workspace


def kcp_compose(transitions, n_prev: int, initial_state=None, *, out=None, stream=None):
    """Step 3: folds maps 0 .. n_prev-1 of the gathered transitions
    ([R, 2, N, H, 128, 128] fp32, device order) over initial_state (fp32
    [N, H, 128, 128] or None = zero).  Returns this device's initial state."""
    torch = _torch()
    _check_cuda(transitions, initial_state, out)
    _, _, N, H, dk, dv = transitions.shape
    s_in = out if out is not None else torch.empty((N, H, dk, dv), dtype=torch.float32, device=transitions.device)
    st = load_library().kda_kcp_compose(_ptr(transitions), int(n_prev), _ptr(initial_state), _ptr(s_in), N, H, dk,
                                        dv, _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_kcp_compose")
    return s_in


def kcp_finish(state_in, workspace, *, shape, dtype, cu_seqlens=None, max_seqlen=None, gate=None, norm_weight=None,
               eps: float = 1e-6, out_dtype=None, output_final_state: bool = True, out=None, stream=None):
    """Step 4: this device's outputs from its initial state and the workspace
    kcp_transition filled.  shape = (B, T, H, 128) and dtype of the segment's
    inputs (the gate's dtype).  Returns (o or y [B, T, H, 128], final_state)."""
    torch = _torch()
    _check_cuda(state_in, workspace, cu_seqlens, gate, norm_weight)
    B, T, H, dv = shape
    if gate is not None and gate.dtype != dtype:
        raise TypeError("the gate must have the inputs' dtype")
    if cu_seqlens is not None:
        if max_seqlen is None:
            raise ValueError("varlen needs max_seqlen (host int)")
        N, maxlen = cu_seqlens.numel() - 1, int(max_seqlen)
    else:
        N, maxlen = B, T
    in_dt = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    odt = out_dtype if out_dtype is not None else dtype
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=odt, device=workspace.device)
    fs = torch.empty((N, H, HEAD_DIM, dv), dtype=torch.float32, device=workspace.device) if output_final_state else None
    st = load_library().kda_kcp_finish(_ptr(state_in), _ptr(o), _ptr(fs), B, T, H, HEAD_DIM, dv, _ptr(cu_seqlens), N,
                                       maxlen, in_dt, _dt(o), _ptr(gate), _ptr(norm_weight), float(eps),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_kcp_finish")
    return o, fs


def decode_step(state, q, k, v, log_alpha, beta, *, scale: float = 1.0, gate=None, norm_weight=None,
                eps: float = 1e-6, out_dtype=None, out=None, stream=None, slots=None):
    """One recurrent step.  state: fp32 [Bd, H, 128, 128] (updated in place);
    q, k, log_alpha, v: [Bd, H, 128]; beta: [Bd, H].  Returns o (or y) [Bd, H, 128].
    slots: int32 [Bd] on the device: the states lie in a pool [P, H, 128, 128], row b's
    in page slots[b]; a negative slot marks a row of padding (also one of P and above,
    and one that an earlier row names): its outputs are zeros and no state changes."""
    torch = _torch()
    if slots is not None:
        one = lambda t: None if t is None else t[None]  # noqa: E731
        o = decode_steps(state, one(q), one(k), one(v), one(log_alpha), one(beta), scale=scale, gate=one(gate),
                         norm_weight=norm_weight, eps=eps, out_dtype=out_dtype, out=one(out), stream=stream,
                         slots=slots)
        return out if out is not None else o[0]
    _check_cuda(state, q, k, v, log_alpha, beta, gate, norm_weight)
    if state.dtype != torch.float32:
        raise TypeError("state must be fp32")
    Bd, H, dk = q.shape
    dv = v.shape[-1]
    odt = out_dtype if out_dtype is not None else q.dtype
    o = out if out is not None else torch.empty((Bd, H, dv), dtype=odt, device=q.device)
    st = load_library().kda_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(o),
                                        Bd, H, dk, dv, _dt(q), _dt(o), float(scale), _ptr(gate), _ptr(norm_weight),
                                        float(eps), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step")
    return o


def decode_steps(state, q, k, v, log_alpha, beta, *, scale: float = 1.0, gate=None, norm_weight=None,
                 eps: float = 1e-6, out_dtype=None, out=None, step_states=None, stream=None, slots=None):
    """n consecutive recurrent steps in one call (e.g. verifying n draft tokens).
    state: fp32 [Bd, H, 128, 128], carried through the steps in place;
    q, k, log_alpha, v: [n, Bd, H, 128]; beta: [n, Bd, H].  step_states: None,
    True (allocate) or an fp32 [n, Bd, H, 128, 128] tensor that receives the state
    after every step.  slots: as decode_step (state is then a pool of pages; with a
    gate, o is normalised in fp32 whatever n is).  Returns o (or y) [n, Bd, H, 128], or
    (o, step_states) when step_states was requested."""
    if slots is not None:
        return _decode_steps_paged(state, slots, q, k, v, log_alpha, beta, scale, gate, norm_weight, eps, out_dtype,
                                   out, step_states, stream)
    torch = _torch()
    want = step_states is not None
    if step_states is True:
        step_states = torch.empty((q.shape[0],) + tuple(state.shape), dtype=torch.float32, device=q.device)
    _check_cuda(state, q, k, v, log_alpha, beta, gate, norm_weight, step_states if want else None)
    if state.dtype != torch.float32:
        raise TypeError("state must be fp32")
    n, Bd, H, dk = q.shape
    dv = v.shape[-1]
    odt = out_dtype if out_dtype is not None else q.dtype
    o = out if out is not None else torch.empty((n, Bd, H, dv), dtype=odt, device=q.device)
    st = load_library().kda_decode_steps(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                         _ptr(o), n, Bd, H, dk, dv, _dt(q), _dt(o), float(scale), _ptr(gate),
                                         _ptr(norm_weight), float(eps), _ptr(step_states if want else None),
                                         _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_steps")
    return (o, step_states) if want else o


def _decode_steps_paged(state, slots, q, k, v, log_alpha, beta, scale, gate, norm_weight, eps, out_dtype, out,
                        step_states, stream):
    torch = _torch()
    _check_cuda(q)
    if q.dim() != 4:
        raise ValueError("q must be [n, Bd, H, 128]")
    there = _elsewhere(q, stream)
    if there is not None:
        with there:
            return _decode_steps_paged(state, slots, q, k, v, log_alpha, beta, scale, gate, norm_weight, eps, out_dtype,
                                       out, step_states, None)
    n, Bd, H, dk = q.shape
    dv = v.shape[-1]
    rows = (n, Bd, H)
    _check_sizes("kda_decode_steps_paged", n, Bd, H, state.shape[0])
    _check_like(q, torch.float32, (state.shape[0], H, dk, dv), "state", state)
    _check_slots(q, slots, "slots", Bd)
    for t, shape, name in ((k, rows + (dk,), "k"), (v, rows + (dv,), "v"), (log_alpha, rows + (dk,), "log_alpha"),
                           (beta, rows, "beta"), (gate, rows + (dv,), "gate")):
        _check_like(q, q.dtype, shape, name, t)
    _check_like(q, torch.float32, (dv,), "norm_weight", norm_weight)
    o, want = out, step_states is not None
    if o is None:
        o = _empty(v, v.shape, out_dtype)
    else:
        _check_like(q, out_dtype if out_dtype is not None else o.dtype, rows + (dv,), "out", o)
    if step_states is True:
        step_states = _empty(q, rows + (dk, dv), torch.float32)
    _check_like(q, torch.float32, rows + (dk, dv), "step_states", step_states)
    st = load_library().kda_decode_steps_paged(_at(state), _at(slots), state.shape[0], _at(q), _at(k), _at(v),
                                               _at(log_alpha), _at(beta), _at(o), n, Bd, H, dk, dv, _dt(q), _dt(o),
                                               scale, _at(gate), _at(norm_weight), eps, _at(step_states),
                                               _here(q.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_steps_paged")
    return (o, step_states) if want else o


def gate_norm(o, g, norm_weight=None, *, eps: float = 1e-6, out_dtype=None, out=None, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * w * sigmoid(g) over the last dim (128)."""
    torch = _torch()
    _check_cuda(o, g, norm_weight)
    dv = o.shape[-1]
    rows = o.numel() // dv
    odt = out_dtype if out_dtype is not None else o.dtype
    y = out if out is not None else torch.empty(o.shape, dtype=odt, device=o.device)
    st = load_library().kda_gate_norm(_ptr(o), _ptr(g), _ptr(norm_weight), float(eps), _ptr(y), rows, dv,
                                      _dt(o), _dt(y), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_gate_norm")
    return y


def _elsewhere(t, stream):
    """None where a call on tensor t can run as things are; else the context for it: its
    device current, and `stream` (of that device) the current stream, so that what the
    call allocates belongs to it."""
    torch = _torch()
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() == torch.cuda.current_device():
        return None
    return torch.cuda.device(t.device)


def _here(device_index):
    """The current stream of the current device, as the library takes it."""
    return _torch()._C._cuda_getCurrentRawStream(device_index)


def _empty(x, shape, dtype):
    """A new contiguous tensor beside x (dtype None: x's)."""
    if shape == x.shape and (dtype is None or dtype == x.dtype) and x.is_contiguous():
        return _torch().empty_like(x)
    return x.new_empty(shape, dtype=dtype)


def _at(t):
    return None if t is None else t.data_ptr()


def _check_sizes(what, *sizes):
    """Sizes that the library takes in 32 bits (ctypes would cut them silently)."""
    if max(sizes) > 0x7FFFFFFF:
        raise KdaError(-2, what)


def _check_like(x, dtype, shape, name, t):
    """t: None, or a contiguous tensor of this dtype and shape on x's device."""
    if t is None or (t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.get_device() == x.get_device()):
        return
    if not t.is_cuda or t.device != x.device:
        raise ValueError(f"{name} must be a CUDA tensor on {x.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check_slots(x, slots, name, n=None):
    torch = _torch()
    if slots is None:
        if n is None:
            raise TypeError(f"{name} must be an int32 vector on the device")
        return
    if not slots.is_cuda or slots.device != x.device:
        raise ValueError(f"{name} must be a CUDA tensor on {x.device}")
    if slots.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    _check_sizes(name, slots.numel())
    if slots.dim() != 1 or (n is not None and slots.numel() != n) or not slots.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector" + (f" of {n}" if n is not None else ""))


def _workspace_bytes(x, workspace):
    if workspace is None:
        return 0
    if not workspace.is_cuda or workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {x.device}")
    return workspace.numel() * workspace.element_size()


def _token_rows(x, t, name):
    """Token stride (elements) of a scan input [B, T, ...] whose channels lie together."""
    if t.device != x.device or not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors on one device (there is no CPU path)")
    if t.dtype != x.dtype:
        raise TypeError("x, log_alpha, gate and d_h must share one dtype")
    if t.shape != x.shape:
        raise ValueError(f"{name} must have x's shape {tuple(x.shape)}, not {tuple(t.shape)}")
    if t.is_contiguous() or t.numel() == 0:
        return 0
    D = 1
    for size, stride in zip(reversed(t.shape[2:]), reversed(t.stride()[2:])):
        if size > 1 and stride != D:
            raise ValueError(f"{name}: the channels of a token must lie together")
        D *= size
    B, T = t.shape[0], t.shape[1]
    row = t.stride(1) if T > 1 else t.stride(0) if B > 1 else D
    if row < D or (B > 1 and T > 1 and t.stride(0) != T * row):
        raise ValueError(f"{name}: tokens must lie at one distance of at least a token's channels")
    return row


def _scan_dims(x, cu_seqlens, initial_state):
    if not x.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    if x.dim() < 3:
        raise ValueError("x must be [B, T, D] (or [B, T, H, d])")
    B, T = x.shape[0], x.shape[1]
    ch = tuple(x.shape[2:])
    N = B
    if cu_seqlens is not None:
        _check_slots(x, cu_seqlens, "cu_seqlens")
        N = cu_seqlens.numel() - 1
    if initial_state is not None:
        _check_like(x, _torch().float32, (N,) + ch, "initial_state", initial_state)
    D = math.prod(ch)
    _check_sizes("kda_scan", B, D, N)
    return B, T, ch, D, N


def scan_fwd(x, log_alpha, initial_state=None, *, gate=None, normalize: bool = False, cu_seqlens=None, out_dtype=None,
             output_final_state: bool = True, final_state=None, out=None, chunk_states=None, workspace=None,
             stream=None):
    """Element-wise gated scan: h_t = a_t h_{t-1} + w_t sigmoid(gate_t) x_t with
    a_t = exp(min(log_alpha_t, 0)), and w_t = sqrt(1 - a_t^2) if normalize else 1.

    x, log_alpha, gate: [B, T, D] or [B, T, H, d] (bf16 or fp32, one dtype; gate
    optional: factor 1).  They may be column slices of wider tensors: the channels of
    a token lie together, the tokens at one distance.  initial_state: fp32 [N, D]
    ([N, H, d]) or None.  Varlen: B = 1 and cu_seqlens int32 [N+1] on the device;
    rows of tokens behind cu_seqlens[N] are left as they are.
    Returns (h, final_state fp32 [N, D] or None); with chunk_states (True: allocate)
    also those, fp32 [ceil(B T / 8), D], for scan_bwd.  workspace: optional, for
    query_status: without it a cu_seqlens that breaks its rules, or a wait on the device that
    gave up, leaves undefined outputs and no trace."""
    torch = _torch()
    B, T, ch, D, N = _scan_dims(x, cu_seqlens, initial_state)
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return scan_fwd(x, log_alpha, initial_state, gate=gate, normalize=normalize, cu_seqlens=cu_seqlens,
                            out_dtype=out_dtype, output_final_state=output_final_state, final_state=final_state,
                            out=out, chunk_states=chunk_states, workspace=workspace)
    ldx, ldl = _token_rows(x, x, "x"), _token_rows(x, log_alpha, "log_alpha")
    ldg = 0 if gate is None else _token_rows(x, gate, "gate")
    h, fs, want = out, final_state, chunk_states is not None
    if h is None:
        h = _empty(x, x.shape, out_dtype)
    else:
        _check_like(x, out_dtype if out_dtype is not None else h.dtype, x.shape, "out", h)
    if fs is not None:
        _check_like(x, torch.float32, (N,) + ch, "final_state", fs)
    elif output_final_state:
        fs = _empty(x, (N,) + ch, torch.float32)
    if want:
        shape = (-(-B * T // SCAN_CHUNK),) + ch
        if chunk_states is True:
            chunk_states = _empty(x, shape, torch.float32)
        _check_like(x, torch.float32, shape, "chunk_states", chunk_states)
    ws_bytes = _workspace_bytes(x, workspace)
    st = load_library().kda_scan_fwd(_at(x), _at(log_alpha), _at(gate), _at(initial_state), _at(h), _at(fs),
                                     _at(chunk_states), B, T, D, ldx, ldl, ldg, _at(cu_seqlens), N, _dt(x), _dt(h),
                                     int(normalize), _at(workspace), ws_bytes,
                                     _here(x.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_scan_fwd")
    return (h, fs, chunk_states) if want else (h, fs)


def scan_bwd_workspace_size(B: int, T: int, D: int) -> int:
    """Workspace bytes of scan_bwd without chunk_states."""
    _check_sizes("kda_scan_bwd_workspace_size", B, D)
    n = ctypes.c_size_t(0)
    st = load_library().kda_scan_bwd_workspace_size(B, T, D, ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_scan_bwd_workspace_size")
    return n.value


def scan_bwd(x, log_alpha, d_h, initial_state=None, d_final_state=None, *, gate=None, normalize: bool = False,
             cu_seqlens=None, chunk_states=None, out_dtype=None, want_d_initial_state: bool = True, workspace=None,
             stream=None):
    """Gradients of scan_fwd: inputs as there, d_h = dL/dh (x's dtype and shape),
    d_final_state = dL/d(final state) fp32 [N, D] or None.  chunk_states: what
    scan_fwd(chunk_states=True) returned for the same inputs; without them they are
    computed first.  Returns a dict: dx, dlog_alpha, dgate (x's shape, fp32 or
    out_dtype; dgate None without a gate) and d_initial_state fp32 [N, D] (None when
    not wanted).  workspace: as scan_fwd; without chunk_states scan_bwd_workspace_size bytes
    (None: allocated, then its status word cannot be asked for)."""
    torch = _torch()
    B, T, ch, D, N = _scan_dims(x, cu_seqlens, initial_state)
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return scan_bwd(x, log_alpha, d_h, initial_state, d_final_state, gate=gate, normalize=normalize,
                            cu_seqlens=cu_seqlens, chunk_states=chunk_states, out_dtype=out_dtype,
                            want_d_initial_state=want_d_initial_state, workspace=workspace)
    ld = (_token_rows(x, x, "x"), _token_rows(x, log_alpha, "log_alpha"),
          0 if gate is None else _token_rows(x, gate, "gate"), _token_rows(x, d_h, "d_h"))
    _check_like(x, torch.float32, (N,) + ch, "d_final_state", d_final_state)
    _check_like(x, torch.float32, (-(-B * T // SCAN_CHUNK),) + ch, "chunk_states", chunk_states)
    odt = out_dtype if out_dtype is not None else torch.float32
    g = {k: _empty(x, x.shape, odt) for k in ("dx", "dlog_alpha")}
    g["dgate"] = None if gate is None else _empty(x, x.shape, odt)
    g["d_initial_state"] = _empty(x, (N,) + ch, torch.float32) if want_d_initial_state else None
    if workspace is None and chunk_states is None:
        workspace = _empty(x, (scan_bwd_workspace_size(B, T, D),), torch.uint8)
    ws_bytes = _workspace_bytes(x, workspace)
    st = load_library().kda_scan_bwd(_at(x), _at(log_alpha), _at(gate), _at(initial_state), _at(d_h),
                                     _at(d_final_state), _at(chunk_states), _at(g["dx"]), _at(g["dlog_alpha"]),
                                     _at(g["dgate"]), _at(g["d_initial_state"]), B, T, D, *ld, _at(cu_seqlens), N,
                                     _dt(x), _dt(g["dx"]), int(normalize), _at(workspace),
                                     ws_bytes, _here(x.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_scan_bwd")
    return g


def scan_decode_steps(state, x, log_alpha, *, gate=None, normalize: bool = False, slots=None, out_dtype=None, out=None,
                      step_states=None, stream=None):
    """n consecutive tokens of the element-wise gated scan for Bd sequences.
    x, log_alpha, gate: contiguous [n, Bd, D] ([n, Bd, H, d]; the prefill alone takes
    columns of wider tensors as they lie).  state: fp32 [P, D], updated in place:
    sequence b's is row slots[b] (int32 [Bd]; None: row b).  A negative slot marks a row
    of padding (also one of P and above, and one that an earlier row names): its outputs
    are zeros and no state changes.  step_states: None, True (allocate) or fp32
    [n, Bd, D] receiving the state after every token.
    Returns h [n, Bd, D], or (h, step_states)."""
    torch = _torch()
    _check_cuda(x)
    if x.dim() < 3:
        raise ValueError("x must be [n, Bd, D] (or [n, Bd, H, d])")
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return scan_decode_steps(state, x, log_alpha, gate=gate, normalize=normalize, slots=slots,
                                     out_dtype=out_dtype, out=out, step_states=step_states)
    shape = x.shape
    _check_like(x, x.dtype, shape, "log_alpha", log_alpha)
    _check_like(x, x.dtype, shape, "gate", gate)
    n, Bd = shape[0], shape[1]
    ch, P = tuple(shape[2:]), state.shape[0]
    D = math.prod(ch)
    _check_sizes("kda_scan_decode_steps", n, Bd, P, D)
    _check_like(x, torch.float32, (P,) + ch, "state", state)
    _check_slots(x, slots, "slots", Bd)
    h, want = out, step_states is not None
    if h is None:
        h = _empty(x, shape, out_dtype)
    else:
        _check_like(x, out_dtype if out_dtype is not None else h.dtype, shape, "out", h)
    if step_states is True:
        step_states = _empty(x, shape, torch.float32)
    _check_like(x, torch.float32, shape, "step_states", step_states)
    st = load_library().kda_scan_decode_steps(_at(state), _at(x), _at(log_alpha), _at(gate), _at(h), _at(slots), P, n,
                                              Bd, D, _dt(x), _dt(h), int(normalize), _at(step_states),
                                              _here(x.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_scan_decode_steps")
    return (h, step_states) if want else h


def scan_decode_step(state, x, log_alpha, *, gate=None, normalize: bool = False, slots=None, out_dtype=None, out=None,
                     stream=None):
    """scan_decode_steps for one token: x, log_alpha, gate [Bd, D]; returns h [Bd, D]."""
    one = lambda t: None if t is None else t[None]  # noqa: E731
    h = scan_decode_steps(state, one(x), one(log_alpha), gate=one(gate), normalize=normalize, slots=slots,
                          out_dtype=out_dtype, out=one(out), stream=stream)
    return out if out is not None else h[0]


@functools.lru_cache(maxsize=64)
def gate_norm_bwd_workspace_size(rows: int) -> int:
    """Workspace bytes of gate_norm_bwd with d_norm_weight."""
    n = ctypes.c_size_t(0)
    st = load_library().kda_gate_norm_bwd_workspace_size(rows, HEAD_DIM, ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_gate_norm_bwd_workspace_size")
    return n.value


def gate_norm_bwd(o, g, d_y, norm_weight=None, *, eps: float = 1e-6, out_dtype=None,
                  want_d_norm_weight: bool = True, workspace=None, stream=None):
    """Gradients of gate_norm: o, g and d_y = dL/dy [..., 128] of one dtype.  Returns a dict:
    d_o, d_gate (o's shape, fp32 or out_dtype) and d_norm_weight fp32 [128] (None when not
    wanted; without a norm_weight the gradient at a weight of ones)."""
    torch = _torch()
    _check_cuda(o)
    if o.shape[-1] != HEAD_DIM:
        raise KdaError(-2, "kda_gate_norm_bwd")
    there = _elsewhere(o, stream)
    if there is not None:
        with there:
            return gate_norm_bwd(o, g, d_y, norm_weight, eps=eps, out_dtype=out_dtype,
                                 want_d_norm_weight=want_d_norm_weight, workspace=workspace)
    _check_like(o, o.dtype, o.shape, "g", g)
    _check_like(o, o.dtype, o.shape, "d_y", d_y)
    _check_like(o, torch.float32, (HEAD_DIM,), "norm_weight", norm_weight)
    rows = o.numel() // HEAD_DIM
    odt = out_dtype if out_dtype is not None else torch.float32
    r = dict(d_o=_empty(o, o.shape, odt), d_gate=_empty(o, o.shape, odt),
             d_norm_weight=_empty(o, (HEAD_DIM,), torch.float32) if want_d_norm_weight else None)
    if workspace is None and want_d_norm_weight:
        workspace = _empty(o, (gate_norm_bwd_workspace_size(rows),), torch.uint8)
    st = load_library().kda_gate_norm_bwd(_at(o), _at(g), _at(d_y), _at(norm_weight), eps, _at(r["d_o"]),
                                          _at(r["d_gate"]), _at(r["d_norm_weight"]), rows, HEAD_DIM, _dt(o),
                                          _dt(r["d_o"]), _at(workspace),
                                          _workspace_bytes(o, workspace), _here(o.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_gate_norm_bwd")
    return r


def _pool_dims(t, layered, name):
    """(layers, pages, bytes of a page, bytes between layers) of a pool [P, ...] or [L, P, ...]."""
    lead = 2 if layered else 1
    if t.dim() < lead:
        raise ValueError(f"{name} must be [{'layers, ' if layered else ''}pages, ...]")
    page = math.prod(t.shape[lead:]) * t.element_size()
    L, P = (t.shape[0], t.shape[1]) if layered else (1, t.shape[0])
    if not t.is_contiguous() and not (layered and L > 0 and t[0].is_contiguous()):
        raise ValueError(f"the pages of {name} must be contiguous, one behind the other")
    return L, P, page, t.stride(0) * t.element_size() if layered else 0


def state_copy(dst, dst_slots, src, src_slots, *, layered: bool = False, stream=None):
    """Copies pages of recurrent states: for each i in list order, dst[dst_slots[i]] =
    src[src_slots[i]], or zeros where src_slots[i] < 0.  dst, src: pools [P, ...] of one
    dtype and page shape (or one pool twice); layered: [L, P, ...], the same slots in
    every layer.  Slots are int32 vectors on the device; an entry with a negative
    destination, or a slot out of range, does nothing.  The result is that of carrying
    the list out one by one.  src None: every entry clears.  Pools of several layers whose
    address ranges interleave (two slices of a wider one) are refused.  Returns dst."""
    if not dst.is_cuda or (src is not None and (not src.is_cuda or src.device != dst.device)):
        raise ValueError("all tensors must be CUDA tensors on one device (there is no CPU path)")
    _check_slots(dst, dst_slots, "dst_slots")
    _check_slots(dst, src_slots, "src_slots", dst_slots.numel())
    there = _elsewhere(dst, stream)
    if there is not None:
        with there:
            return state_copy(dst, dst_slots, src, src_slots, layered=layered)
    L, P, page, d_layer = _pool_dims(dst, layered, "dst")
    Q, s_layer = 0, 0
    if src is dst:
        Q, s_layer = P, d_layer
    elif src is not None:
        if src.dtype != dst.dtype or src.shape[1 + layered:] != dst.shape[1 + layered:] or \
                (layered and src.shape[0] != L):
            raise ValueError("dst and src must have one dtype, page shape and number of layers")
        _, Q, _, s_layer = _pool_dims(src, layered, "src")
    if page == 0:
        return dst
    _check_sizes("kda_state_copy", L, P, Q)
    lib, n, here = load_library(), dst_slots.numel(), _here(dst.get_device())
    for at in range(0, n, COPY_LIST):  # longer lists in pieces, one behind the other
        d, s = (dst_slots, src_slots) if n <= COPY_LIST else (v[at:at + COPY_LIST] for v in (dst_slots, src_slots))
        st = lib.kda_state_copy(_at(dst), _at(src), L, page, P, Q, d_layer, s_layer, _at(d), _at(s), d.numel(), here)
        if st != KDA_OK:
            raise KdaError(st, "kda_state_copy")
    return dst


def _check_live(live):
    torch = _torch()
    _check_cuda(live)
    if live.dtype not in (torch.uint8, torch.bool) or live.dim() != 1:
        raise TypeError("live must be a vector of uint8 or bool, one per page")
    _check_sizes("live", live.numel())


def state_alloc(live, n: int, *, stream=None):
    """Takes the n lowest free slots of a pool: marks them in live (uint8 or bool [P], on the
    device) and returns them as int32 [n], -1 where no slot was left."""
    torch = _torch()
    _check_live(live)
    _check_sizes("kda_state_alloc", n)
    there = _elsewhere(live, stream)
    if there is not None:
        with there:
            return state_alloc(live, n)
    slots = _empty(live, (n,), torch.int32)
    st = load_library().kda_state_alloc(_at(live), live.numel(), _at(slots), n, _here(live.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_state_alloc")
    return slots


def state_free(live, slots, *, stream=None):
    """Marks slots (int32, on the device; those out of range are ignored) free in live."""
    _check_live(live)
    _check_slots(live, slots, "slots")
    there = _elsewhere(live, stream)
    if there is not None:
        with there:
            return state_free(live, slots)
    st = load_library().kda_state_free(_at(live), live.numel(), _at(slots), slots.numel(), _here(live.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_state_free")


def state_compact(live, *, stream=None):
    """Plans the moves that bring the live pages of a pool to its front and updates live.
    Returns a dict of int32 tensors: dst_slots, src_slots [P] (the moves, then -1: pass
    both to state_copy with the pool twice, for every pool that shares the slots),
    new_slots [P] (where each old slot's page lies now, -1 if free) and n_live [1]."""
    torch = _torch()
    _check_live(live)
    there = _elsewhere(live, stream)
    if there is not None:
        with there:
            return state_compact(live)
    P = live.numel()
    parts = _empty(live, (3 * P + 1,), torch.int32).split((P, P, P, 1))  # one allocation
    r = dict(zip(("dst_slots", "src_slots", "new_slots", "n_live"), parts))
    st = load_library().kda_state_compact(_at(live), P, _at(r["dst_slots"]), _at(r["src_slots"]), _at(r["new_slots"]),
                                          _at(r["n_live"]), _here(live.get_device()))
    if st != KDA_OK:
        raise KdaError(st, "kda_state_compact")
    return r


def query_status(workspace, stream=None) -> int:
    """Synchronises, returns and clears the device status word of a workspace."""
    return load_library().kda_query_status(_ptr(workspace), _stream(stream))


def profile_enable(on: bool = True) -> None:
    """Per-kernel device timing of later library launches (CUDA events)."""
    load_library().kda_profile_enable(int(bool(on)))


def profile_read() -> dict:
    """{kernel name: (launches, summed device ms)} since the last read."""
    arr = (KernelTime * 16)()
    n = ctypes.c_int(0)
    st = load_library().kda_profile_read(arr, 16, ctypes.byref(n))
    if st != KDA_OK:
        raise KdaError(st, "kda_profile_read")
    return {arr[i].name.decode(): (arr[i].launches, arr[i].ms) for i in range(min(n.value, 16))}
