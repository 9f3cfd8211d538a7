"""Thin ctypes binding of libkda.so (see include/kda.h).

Argument marshalling only: every function here passes device pointers, sizes
and the current CUDA stream to the C ABI, and every step of the computation
runs in the library's CUDA kernels.  There is no CPU fallback: if libkda.so
cannot be loaded, every call raises :class:`KdaError`.

Functions with the C names take tensors that are already allocated (device
tensors from PyTorch) and return the status code, raising :class:`KdaError`
on anything but ``KDA_OK`` unless ``check=False``.  :func:`chunk_fwd` and
:func:`decode_step` are convenience wrappers that allocate outputs and the
workspace with PyTorch and then make the same calls.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_TIMEOUT = 4
KDA_ERR_WORKSPACE = 5
KDA_ERR_BAD_SEQLENS = 6

KDA_DTYPE_F32 = 0
KDA_DTYPE_BF16 = 1

# Every symbol include/kda.h declares.
EXPORTS = (
    "kda_status_string", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd",
    "kda_num_chunks_upper_bound", "kda_chunk_gate_cumsum", "kda_chunk_intra",
    "kda_chunk_inter", "kda_chunk_output", "kda_decode_step", "kda_get_device_status",
    "kda_chunk_fwd_noalloc", "kda_chunk_split_workspace_size", "kda_chunk_split_intra",
    "kda_chunk_split_chain", "kda_chunk_fwd_plan", "kda_qkv_conv_norm",
    "kda_output_norm_gate", "kda_gdn_chunk_fwd_workspace_size", "kda_gdn_chunk_fwd",
    "kda_gdn_decode_step", "kda_chunk_bwd_workspace_size", "kda_chunk_bwd",
    "kda_gdn_chunk_bwd_workspace_size", "kda_gdn_chunk_bwd", "kda_qkv_conv_norm_step",
    "kda_chunk_fwd_with_plan", "kda_chunk_fwd_plan_workspace_size",
    "kda_test_overlap_flag_timeout", "kda_layer_decode_step", "kda_layer_chunk_fwd",
    "kda_layer_chunk_fwd_workspace_size", "kda_chunk_state_maps", "kda_fold_segment_states",
    "kda_linear_scan_num_entries", "kda_linear_scan_workspace_size",
    "kda_linear_scan_bwd_workspace_size", "kda_linear_scan_fwd", "kda_linear_scan_bwd",
    "kda_linear_scan_step", "kda_fp8_pitch", "kda_add_rms_norm",
    "kda_add_rms_norm_bwd_workspace_size", "kda_add_rms_norm_bwd", "kda_quantize_fp8",
    "kda_fp8_matmul", "kda_test_linear_scan_timeout", "kda_test_fp8_matmul_timeout", "kda_test_fp8_matmul_plan",
)


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {status_string(status)}" if what else status_string(status))


_lib = None
_lock = threading.Lock()

_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "kda_status_string": ([_i], ctypes.c_char_p),
    "kda_chunk_fwd_workspace_size": ([_i, _i, _i, _i, _i, _i, _i], _sz),
    "kda_num_chunks_upper_bound": ([_i, _i, _i], _i),
    "kda_chunk_fwd": ([_vp] * 7 + [_i] * 8 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_chunk_gate_cumsum": ([_vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp], _i),
    "kda_chunk_intra": ([_vp] * 5 + [_i] * 8 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_chunk_inter": ([_vp] * 6 + [_i] * 8 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_chunk_output": ([_vp] * 6 + [_i] * 8 + [_vp, _vp, _sz, _vp], _i),
    "kda_decode_step": ([_vp] * 7 + [_i] * 5 + [_vp], _i),
    "kda_get_device_status": ([_vp, _vp], _i),
    "kda_chunk_fwd_noalloc": ([_vp] * 7 + [_i] * 8 + [_vp, _vp, _vp], _i),
    "kda_chunk_split_workspace_size": ([_i, _i, _i], _sz),
    "kda_chunk_fwd_plan": ([_i] * 8, _i),
    "kda_chunk_fwd_with_plan": ([_i] + [_vp] * 7 + [_i] * 8 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_chunk_fwd_plan_workspace_size": ([_i] * 8, _sz),
    "kda_test_overlap_flag_timeout": ([_vp] * 7 + [_i] * 4 + [_vp] * 3 + [_sz, _i, _i,
                                      ctypes.c_ulonglong, _vp], _i),
    "kda_qkv_conv_norm": ([_vp] * 7 + [_i] * 7 + [ctypes.c_float] + [_vp] * 4, _i),
    "kda_output_norm_gate": ([_vp] * 3 + [_i] * 4 + [ctypes.c_float] + [_vp] * 2, _i),
    "kda_gdn_chunk_fwd_workspace_size": ([_i] * 7, _sz),
    "kda_gdn_chunk_fwd": ([_vp] * 7 + [_i] * 8 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_gdn_decode_step": ([_vp] * 7 + [_i] * 5 + [_vp], _i),
    "kda_chunk_bwd_workspace_size": ([_i] * 5, _sz),
    "kda_chunk_bwd": ([_vp] * 9 + [_i] * 7 + [_vp] * 7 + [_sz, _vp], _i),
    "kda_gdn_chunk_bwd_workspace_size": ([_i] * 5, _sz),
    "kda_gdn_chunk_bwd": ([_vp] * 9 + [_i] * 7 + [_vp] * 7 + [_sz, _vp], _i),
    "kda_qkv_conv_norm_step": ([_vp] * 9 + [_i] * 5 + [ctypes.c_float] + [_vp] * 4, _i),
    "kda_chunk_split_intra": ([_vp] * 5 + [_i] * 4 + [_vp, _sz, _vp], _i),
    "kda_layer_decode_step": ([_vp] * 14 + [_i] * 5 + [ctypes.c_float] * 2 + [_vp, _vp], _i),
    "kda_layer_chunk_fwd": ([_vp] * 10 + [_i] * 8 + [_vp, _vp] + [ctypes.c_float] * 2 +
                            [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_layer_chunk_fwd_workspace_size": ([_i] * 7, _sz),
    "kda_chunk_state_maps": ([_vp] * 6 + [_i] * 4 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_fold_segment_states": ([_vp] * 3 + [_i] * 6 + [_vp, _vp, _vp], _i),
    "kda_chunk_split_chain": ([_vp] * 3 + [_i] * 4 + [_vp, _vp, _vp, _sz, _vp], _i),
    "kda_linear_scan_num_entries": ([_i], _i),
    "kda_linear_scan_workspace_size": ([_i] * 3, _sz),
    "kda_linear_scan_bwd_workspace_size": ([_i] * 3, _sz),
    "kda_linear_scan_fwd": ([_vp] * 4 + [_i] * 6 + [_vp] * 4 + [_sz, _vp], _i),
    "kda_linear_scan_bwd": ([_vp] * 7 + [_i] * 6 + [_vp] * 4 + [_sz, _vp], _i),
    "kda_linear_scan_step": ([_vp] * 5 + [_i] * 4 + [_vp], _i),
    "kda_fp8_pitch": ([_i], _i),
    "kda_add_rms_norm": ([_vp] * 3 + [_i] * 3 + [ctypes.c_float] + [_vp] * 5, _i),
    "kda_add_rms_norm_bwd_workspace_size": ([_i] * 2, _sz),
    "kda_add_rms_norm_bwd": ([_vp] * 4 + [_i] * 3 + [ctypes.c_float] + [_vp] * 3 + [_sz, _vp], _i),
    "kda_quantize_fp8": ([_vp] + [_i] * 5 + [_vp] * 3, _i),
    "kda_fp8_matmul": ([_vp] * 4 + [_i] * 5 + [_vp] * 2, _i),
    "kda_test_linear_scan_timeout": ([_vp] * 4 + [_i] * 4 + [_vp] * 3 +
                                     [_sz, ctypes.c_ulonglong, _vp], _i),
    "kda_test_fp8_matmul_timeout": ([_vp] * 4 + [_i] * 5 + [_vp] + [_i] * 2 + [_vp], _i),
    "kda_test_fp8_matmul_plan": ([_i] * 5 + [_vp] * 2, _i),
}

# Size of the library's built-in scratch used by kda_chunk_fwd_noalloc.
KDA_NOALLOC_SCRATCH_BYTES = 64 << 20


def load(path: str = LIB_PATH):
    """Load libkda.so (once).  Raises KdaError if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise KdaError(KDA_ERR_CUDA, f"libkda.so not found at {path}; run "
                               "`python -m gated_delta_rule_124_b200.build`")
            lib = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load().kda_status_string(int(status)).decode()
    except KdaError:
        return f"status {status}"


def _p(t) -> int | None:
    """Device pointer of a tensor (or None for NULL); a plain int is passed
    through as a raw address."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_TORCH_OF = {KDA_DTYPE_F32: torch.float32, KDA_DTYPE_BF16: torch.bfloat16}


def _check(what, dtype=None, typed=(), f32=(), i32=(), raw=()):
    """Reject tensors the C ABI would misread, before any pointer is passed:
    every tensor must be contiguous and on one device; `typed` tensors (q, k,
    v, o, dout ...) must have the call's dtype, `f32` ones (g, beta, states,
    gradients) float32, `i32` ones (cu_seqlens) int32; `raw` ones (workspaces)
    only contiguous.  Plain ints (raw addresses) and None are not checked."""
    want = None if dtype is None else _TORCH_OF[dtype_code(dtype)]
    dev = None
    for group, need in ((typed, want), (f32, torch.float32), (i32, torch.int32), (raw, None)):
        for t in group:
            if t is None or isinstance(t, int):
                continue
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"{what}: expected a tensor, got {type(t).__name__}")
            if not t.is_contiguous():
                raise ValueError(f"{what}: every tensor must be contiguous (got strides "
                                 f"{tuple(t.stride())} for shape {tuple(t.shape)})")
            if need is not None and t.dtype != need:
                raise ValueError(f"{what}: expected {need}, got {t.dtype}")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"{what}: tensors on {dev} and {t.device}")


def _stream(stream) -> int | None:
    if stream is None:
        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_F32, _I32, _ANY = (torch.float32,), (torch.int32,), None
_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _args(what, *pairs):
    """The device pointers of (tensor, the dtypes it may have) pairs, and the index
    of the tensors' device: _check's rules in one pass, for calls short enough
    that a decode step waits for the host.  None and raw addresses pass through."""
    device, out = None, []
    for t, need in pairs:
        if t is None or isinstance(t, int):
            out.append(t)
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{what}: expected a tensor, got {type(t).__name__}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: every tensor must be contiguous (got strides "
                             f"{tuple(t.stride())} for shape {tuple(t.shape)})")
        if need is not None and t.dtype not in need:
            raise ValueError(f"{what}: expected {' or '.join(map(str, need))}, got {t.dtype}")
        d = t.get_device()
        if device is None:
            device = d
        elif d != device:
            raise ValueError(f"{what}: tensors on different devices ({device} and {d})")
        out.append(t.data_ptr())
    if device is not None and device < 0:
        raise ValueError(f"{what}: the tensors are not on a GPU")
    return out, device


# The handle of a device's current stream (without the object around it, where
# this torch offers that).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
# The current device, once there are tensors on one.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(name, device, stream, check, *args) -> int:
    """The library's call `name` with `args` and a stream: the given one, or the
    current stream of the tensors' device, which is the current device during the
    call."""
    fn = getattr(_lib or load(), name)
    if device is None:   # raw addresses
        return _ret(fn(*args, _stream(stream)), name, check)
    if stream is None:
        stream = _current_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == _current_device():
        return _ret(fn(*args, stream), name, check)
    with torch.cuda.device(device):
        return _ret(fn(*args, stream), name, check)


def _used_on(stream, *tensors) -> None:
    """Tensors allocated here for work on a stream of the caller's: their memory
    is not reused before that work is done."""
    if stream is None:
        return
    for t in tensors:
        if t is not None and t.is_cuda:
            s = (torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int)
                 else stream)
            t.record_stream(s)


def dtype_code(dtype) -> int:
    if dtype in (torch.bfloat16, "bf16", KDA_DTYPE_BF16):
        return KDA_DTYPE_BF16
    if dtype in (torch.float32, "f32", KDA_DTYPE_F32):
        return KDA_DTYPE_F32
    raise ValueError(f"unsupported dtype {dtype}")


def _ret(st: int, what: str, check: bool) -> int:
    if check and st != KDA_OK:
        raise KdaError(st, what)
    return st


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------- C-named calls

def kda_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk, dtype) -> int:
    return int(load().kda_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk,
                                                   dtype_code(dtype)))


KDA_PLAN_SIMT, KDA_PLAN_SPLIT, KDA_PLAN_OVERLAP = 0, 2, 3
PLAN_NAMES = {KDA_PLAN_SIMT: "simt", KDA_PLAN_SPLIT: "split", KDA_PLAN_OVERLAP: "overlap"}
PLAN_CODES = {v: k for k, v in PLAN_NAMES.items()}


def plan_code(plan) -> int:
    return PLAN_CODES[plan] if isinstance(plan, str) else int(plan)


def kda_chunk_fwd_plan(total_tokens, num_seqs, H, dk, dv, chunk, dtype, packed=False) -> int:
    return int(load().kda_chunk_fwd_plan(total_tokens, num_seqs, int(bool(packed)), H, dk, dv,
                                         chunk, dtype_code(dtype)))


def kda_num_chunks_upper_bound(total_tokens, num_seqs, chunk) -> int:
    return int(load().kda_num_chunks_upper_bound(total_tokens, num_seqs, chunk))


def kda_chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens, B, T, num_seqs, H, dk, dv,
                  chunk, dtype, o, final_state, workspace, workspace_bytes=None, stream=None,
                  check=True) -> int:
    _check("kda_chunk_fwd", dtype, typed=(q, k, v, o), f32=(g, beta, initial_state, final_state),
           i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(initial_state),
                              _p(cu_seqlens), B, T, num_seqs, H, dk, dv, chunk,
                              dtype_code(dtype), _p(o), _p(final_state), _p(workspace), wb,
                              _stream(stream))
    return _ret(st, "kda_chunk_fwd", check)


def kda_chunk_fwd_plan_workspace_size(plan, total_tokens, num_seqs, H, dk, dv, chunk,
                                      dtype) -> int:
    return int(load().kda_chunk_fwd_plan_workspace_size(plan_code(plan), total_tokens, num_seqs,
                                                        H, dk, dv, chunk, dtype_code(dtype)))


def kda_chunk_fwd_with_plan(plan, q, k, v, g, beta, initial_state, cu_seqlens, B, T, num_seqs, H,
                            dk, dv, chunk, dtype, o, final_state, workspace, workspace_bytes=None,
                            stream=None, check=True) -> int:
    """kda_chunk_fwd on an explicitly chosen plan ('simt', 'split', 'overlap'
    or its KDA_PLAN_* code); KDA_ERR_UNSUPPORTED where it cannot run."""
    _check("kda_chunk_fwd_with_plan", dtype, typed=(q, k, v, o),
           f32=(g, beta, initial_state, final_state), i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_fwd_with_plan(plan_code(plan), _p(q), _p(k), _p(v), _p(g), _p(beta),
                                        _p(initial_state), _p(cu_seqlens), B, T, num_seqs, H,
                                        dk, dv, chunk, dtype_code(dtype), _p(o),
                                        _p(final_state), _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_chunk_fwd_with_plan", check)


def kda_test_overlap_flag_timeout(q, k, v, g, beta, initial_state, cu_seqlens, B, T, num_seqs,
                                  H, o, final_state, workspace, withheld_chunk, withheld_head,
                                  flag_wait_ns, workspace_bytes=None, stream=None,
                                  check=True) -> int:
    """The overlap plan with one chunk's ready flag withheld and the chains'
    flag waits bounded by flag_wait_ns: exercises the bounded-wait error path
    (kda_get_device_status then reports KDA_ERR_TIMEOUT).  Testing only."""
    _check("kda_test_overlap_flag_timeout", "bf16", typed=(q, k, v, o),
           f32=(g, beta, initial_state, final_state), i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_test_overlap_flag_timeout(_p(q), _p(k), _p(v), _p(g), _p(beta),
                                              _p(initial_state), _p(cu_seqlens), B, T, num_seqs,
                                              H, _p(o), _p(final_state), _p(workspace), wb,
                                              withheld_chunk, withheld_head, flag_wait_ns,
                                              _stream(stream))
    return _ret(st, "kda_test_overlap_flag_timeout", check)


def kda_chunk_gate_cumsum(g, cu_seqlens, B, T, num_seqs, H, dk, chunk, G, workspace,
                          workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_gate_cumsum", None, f32=(g, G), i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_gate_cumsum(_p(g), _p(cu_seqlens), B, T, num_seqs, H, dk, chunk,
                                      _p(G), _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_chunk_gate_cumsum", check)


def kda_chunk_intra(k, v, G, beta, cu_seqlens, B, T, num_seqs, H, dk, dv, chunk, dtype, W, Ut,
                    workspace, workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_intra", dtype, typed=(k, v), f32=(G, beta, W, Ut), i32=(cu_seqlens,),
           raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_intra(_p(k), _p(v), _p(G), _p(beta), _p(cu_seqlens), B, T, num_seqs,
                                H, dk, dv, chunk, dtype_code(dtype), _p(W), _p(Ut),
                                _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_chunk_intra", check)


def kda_chunk_inter(k, G, W, U, initial_state, cu_seqlens, B, T, num_seqs, H, dk, dv, chunk,
                    dtype, chunk_states, final_state, workspace, workspace_bytes=None,
                    stream=None, check=True) -> int:
    _check("kda_chunk_inter", dtype, typed=(k,), f32=(G, W, U, initial_state, chunk_states,
           final_state), i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_inter(_p(k), _p(G), _p(W), _p(U), _p(initial_state), _p(cu_seqlens),
                                B, T, num_seqs, H, dk, dv, chunk, dtype_code(dtype),
                                _p(chunk_states), _p(final_state), _p(workspace), wb,
                                _stream(stream))
    return _ret(st, "kda_chunk_inter", check)


def kda_chunk_output(q, k, G, U, chunk_states, cu_seqlens, B, T, num_seqs, H, dk, dv, chunk,
                     dtype, o, workspace, workspace_bytes=None, stream=None,
                     check=True) -> int:
    _check("kda_chunk_output", dtype, typed=(q, k, o), f32=(G, U, chunk_states),
           i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_output(_p(q), _p(k), _p(G), _p(U), _p(chunk_states), _p(cu_seqlens),
                                 B, T, num_seqs, H, dk, dv, chunk, dtype_code(dtype), _p(o),
                                 _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_chunk_output", check)


def kda_chunk_split_workspace_size(total_tokens, num_seqs, H) -> int:
    return int(load().kda_chunk_split_workspace_size(total_tokens, num_seqs, H))


def kda_chunk_split_intra(q, k, g, beta, cu_seqlens, B, T, num_seqs, H, workspace,
                          workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_split_intra", "bf16", typed=(q, k), f32=(g, beta), i32=(cu_seqlens,),
           raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_split_intra(_p(q), _p(k), _p(g), _p(beta), _p(cu_seqlens), B, T,
                                      num_seqs, H, _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_chunk_split_intra", check)


def kda_chunk_split_chain(v, initial_state, cu_seqlens, B, T, num_seqs, H, o, final_state,
                          workspace, workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_split_chain", "bf16", typed=(v, o), f32=(initial_state, final_state),
           i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_split_chain(_p(v), _p(initial_state), _p(cu_seqlens), B, T,
                                      num_seqs, H, _p(o), _p(final_state), _p(workspace), wb,
                                      _stream(stream))
    return _ret(st, "kda_chunk_split_chain", check)


def kda_gdn_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk, dtype) -> int:
    return int(load().kda_gdn_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk,
                                                       dtype_code(dtype)))


def kda_gdn_chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens, B, T, num_seqs, H, dk, dv,
                      chunk, dtype, o, final_state, workspace, workspace_bytes=None, stream=None,
                      check=True) -> int:
    _check("kda_gdn_chunk_fwd", dtype, typed=(q, k, v, o), f32=(g, beta, initial_state,
           final_state), i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_gdn_chunk_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(initial_state),
                                  _p(cu_seqlens), B, T, num_seqs, H, dk, dv, chunk,
                                  dtype_code(dtype), _p(o), _p(final_state), _p(workspace), wb,
                                  _stream(stream))
    return _ret(st, "kda_gdn_chunk_fwd", check)


def kda_gdn_decode_step(q, k, v, g, beta, state, o, N, H, dk, dv, dtype, stream=None,
                        check=True) -> int:
    _check("kda_gdn_decode_step", dtype, typed=(q, k, v, o), f32=(g, beta, state))
    st = load().kda_gdn_decode_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), _p(o), N,
                                    H, dk, dv, dtype_code(dtype), _stream(stream))
    return _ret(st, "kda_gdn_decode_step", check)


def kda_chunk_bwd_workspace_size(total_tokens, num_seqs, H, dk, dv) -> int:
    return int(load().kda_chunk_bwd_workspace_size(total_tokens, num_seqs, H, dk, dv))


def kda_chunk_bwd(q, k, v, g, beta, initial_state, dout, dfinal_state, cu_seqlens, B, T,
                  num_seqs, H, dk, dv, dtype, dq, dk_out, dv_out, dg, dbeta, dinitial_state,
                  workspace, workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_bwd", dtype, typed=(q, k, v, dout), f32=(g, beta, initial_state,
           dfinal_state, dq, dk_out, dv_out, dg, dbeta, dinitial_state), i32=(cu_seqlens,),
           raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_bwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(initial_state),
                              _p(dout), _p(dfinal_state), _p(cu_seqlens), B, T, num_seqs, H, dk,
                              dv, dtype_code(dtype), _p(dq), _p(dk_out), _p(dv_out), _p(dg),
                              _p(dbeta), _p(dinitial_state), _p(workspace), wb,
                              _stream(stream))
    return _ret(st, "kda_chunk_bwd", check)


def kda_gdn_chunk_bwd_workspace_size(total_tokens, num_seqs, H, dk, dv) -> int:
    return int(load().kda_gdn_chunk_bwd_workspace_size(total_tokens, num_seqs, H, dk, dv))


def kda_gdn_chunk_bwd(q, k, v, g, beta, initial_state, dout, dfinal_state, cu_seqlens, B, T,
                      num_seqs, H, dk, dv, dtype, dq, dk_out, dv_out, dg, dbeta, dinitial_state,
                      workspace, workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_gdn_chunk_bwd", dtype, typed=(q, k, v, dout), f32=(g, beta, initial_state,
           dfinal_state, dq, dk_out, dv_out, dg, dbeta, dinitial_state), i32=(cu_seqlens,),
           raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_gdn_chunk_bwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(initial_state),
                                  _p(dout), _p(dfinal_state), _p(cu_seqlens), B, T, num_seqs, H,
                                  dk, dv, dtype_code(dtype), _p(dq), _p(dk_out), _p(dv_out),
                                  _p(dg), _p(dbeta), _p(dinitial_state), _p(workspace), wb,
                                  _stream(stream))
    return _ret(st, "kda_gdn_chunk_bwd", check)


def kda_qkv_conv_norm_step(xq, xk, xv, wq, wk, wv, conv_q, conv_k, conv_v, N, H, dk, dv,
                           dtype, eps, q, k, v, stream=None, check=True) -> int:
    _check("kda_qkv_conv_norm_step", dtype, typed=(xq, xk, xv, conv_q, conv_k, conv_v, q, k, v),
           f32=(wq, wk, wv))
    st = load().kda_qkv_conv_norm_step(_p(xq), _p(xk), _p(xv), _p(wq), _p(wk), _p(wv),
                                       _p(conv_q), _p(conv_k), _p(conv_v), N, H, dk, dv,
                                       dtype_code(dtype), eps, _p(q), _p(k), _p(v),
                                       _stream(stream))
    return _ret(st, "kda_qkv_conv_norm_step", check)


def kda_qkv_conv_norm(xq, xk, xv, wq, wk, wv, cu_seqlens, B, T, num_seqs, H, dk, dv, dtype,
                      eps, q, k, v, stream=None, check=True) -> int:
    _check("kda_qkv_conv_norm", dtype, typed=(xq, xk, xv, q, k, v), f32=(wq, wk, wv),
           i32=(cu_seqlens,))
    st = load().kda_qkv_conv_norm(_p(xq), _p(xk), _p(xv), _p(wq), _p(wk), _p(wv),
                                  _p(cu_seqlens), B, T, num_seqs, H, dk, dv, dtype_code(dtype),
                                  float(eps), _p(q), _p(k), _p(v), _stream(stream))
    return _ret(st, "kda_qkv_conv_norm", check)


def kda_output_norm_gate(o, gate, w, total_tokens, H, dv, dtype, eps, y, stream=None,
                         check=True) -> int:
    _check("kda_output_norm_gate", dtype, typed=(o, gate, y), f32=(w,))
    st = load().kda_output_norm_gate(_p(o), _p(gate), _p(w), total_tokens, H, dv,
                                     dtype_code(dtype), float(eps), _p(y), _stream(stream))
    return _ret(st, "kda_output_norm_gate", check)


def kda_chunk_state_maps(q, k, v, g, beta, cu_seqlens, B, T, num_seqs, H, M, Bm, workspace,
                         workspace_bytes=None, stream=None, check=True) -> int:
    _check("kda_chunk_state_maps", "bf16", typed=(q, k, v), f32=(g, beta, M, Bm),
           i32=(cu_seqlens,), raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_chunk_state_maps(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(cu_seqlens), B, T,
                                     num_seqs, H, _p(M), _p(Bm), _p(workspace), wb,
                                     _stream(stream))
    return _ret(st, "kda_chunk_state_maps", check)


def kda_fold_segment_states(M, Bm, S0, R, N, H, dk, dv, reverse, each, final_state, stream=None,
                            check=True) -> int:
    _check("kda_fold_segment_states", None, f32=(M, Bm, S0, each, final_state))
    st = load().kda_fold_segment_states(_p(M), _p(Bm), _p(S0), R, N, H, dk, dv, int(bool(reverse)),
                                        _p(each), _p(final_state), _stream(stream))
    return _ret(st, "kda_fold_segment_states", check)


def kda_layer_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk, dtype) -> int:
    return int(load().kda_layer_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk,
                                                         dtype_code(dtype)))


def kda_layer_chunk_fwd(xq, xk, xv, wq, wk, wv, g, beta, initial_state, cu_seqlens, B, T,
                        num_seqs, H, dk, dv, chunk, dtype, gate, w_norm, l2_eps, rms_eps, y,
                        final_state, workspace, workspace_bytes=None, stream=None,
                        check=True) -> int:
    _check("kda_layer_chunk_fwd", dtype, typed=(xq, xk, xv, gate, y),
           f32=(wq, wk, wv, g, beta, initial_state, w_norm, final_state), i32=(cu_seqlens,),
           raw=(workspace,))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    st = load().kda_layer_chunk_fwd(_p(xq), _p(xk), _p(xv), _p(wq), _p(wk), _p(wv), _p(g),
                                    _p(beta), _p(initial_state), _p(cu_seqlens), B, T, num_seqs,
                                    H, dk, dv, chunk, dtype_code(dtype), _p(gate), _p(w_norm),
                                    float(l2_eps), float(rms_eps), _p(y), _p(final_state),
                                    _p(workspace), wb, _stream(stream))
    return _ret(st, "kda_layer_chunk_fwd", check)


def kda_layer_decode_step(xq, xk, xv, wq, wk, wv, conv_q, conv_k, conv_v, g, beta, state, gate,
                          w_norm, N, H, dk, dv, dtype, l2_eps, rms_eps, y, stream=None,
                          check=True) -> int:
    _check("kda_layer_decode_step", dtype, typed=(xq, xk, xv, conv_q, conv_k, conv_v, gate, y),
           f32=(wq, wk, wv, g, beta, state, w_norm))
    st = load().kda_layer_decode_step(_p(xq), _p(xk), _p(xv), _p(wq), _p(wk), _p(wv),
                                      _p(conv_q), _p(conv_k), _p(conv_v), _p(g), _p(beta),
                                      _p(state), _p(gate), _p(w_norm), N, H, dk, dv,
                                      dtype_code(dtype), float(l2_eps), float(rms_eps), _p(y),
                                      _stream(stream))
    return _ret(st, "kda_layer_decode_step", check)


def kda_decode_step(q, k, v, g, beta, state, o, N, H, dk, dv, dtype, stream=None,
                    check=True) -> int:
    _check("kda_decode_step", dtype, typed=(q, k, v, o), f32=(g, beta, state))
    st = load().kda_decode_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), _p(o), N, H,
                                dk, dv, dtype_code(dtype), _stream(stream))
    return _ret(st, "kda_decode_step", check)


@functools.lru_cache(maxsize=256)
def kda_linear_scan_num_entries(total_tokens) -> int:
    return int(load().kda_linear_scan_num_entries(total_tokens))


@functools.lru_cache(maxsize=256)
def kda_linear_scan_workspace_size(total_tokens, H, d) -> int:
    return int(load().kda_linear_scan_workspace_size(total_tokens, H, d))


@functools.lru_cache(maxsize=256)
def kda_linear_scan_bwd_workspace_size(total_tokens, H, d) -> int:
    return int(load().kda_linear_scan_bwd_workspace_size(total_tokens, H, d))


def kda_linear_scan_fwd(x, g, initial_state, cu_seqlens, B, T, num_seqs, H, d, dtype, h,
                        final_state, entry_states, workspace, workspace_bytes=None, stream=None,
                        check=True) -> int:
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (px, pg, ph0, pcu, ph, pf, pe, pw), dev = _args(
        "kda_linear_scan_fwd", (x, typed), (g, _F32), (initial_state, _F32), (cu_seqlens, _I32),
        (h, typed), (final_state, _F32), (entry_states, _F32), (workspace, _ANY))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _enqueue("kda_linear_scan_fwd", dev, stream, check, px, pg, ph0, pcu, B, T, num_seqs,
                    H, d, code, ph, pf, pe, pw, wb)


def kda_linear_scan_bwd(x, g, initial_state, dout, dfinal_state, entry_states, cu_seqlens, B, T,
                        num_seqs, H, d, dtype, dx, dg, dinitial_state, workspace,
                        workspace_bytes=None, stream=None, check=True) -> int:
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (px, pg, ph0, pdo, pdf, pe, pcu, pdx, pdg, pdh, pw), dev = _args(
        "kda_linear_scan_bwd", (x, typed), (g, _F32), (initial_state, _F32), (dout, typed),
        (dfinal_state, _F32), (entry_states, _F32), (cu_seqlens, _I32), (dx, typed), (dg, _F32),
        (dinitial_state, _F32), (workspace, _ANY))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _enqueue("kda_linear_scan_bwd", dev, stream, check, px, pg, ph0, pdo, pdf, pe, pcu, B,
                    T, num_seqs, H, d, code, pdx, pdg, pdh, pw, wb)


def kda_test_linear_scan_timeout(x, g, dout, entry_states, T, H, d, dtype, out, dg, workspace,
                                 wait_ns, workspace_bytes=None, stream=None, check=True) -> int:
    """The recurrence (dout None) or its backward with one tile never run and the
    waits for tiles bounded by wait_ns: exercises the bounded-wait error path
    (kda_get_device_status then reports KDA_ERR_TIMEOUT).  Testing only."""
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (px, pg, pd, pe, po, pdg, pw), dev = _args(
        "kda_test_linear_scan_timeout", (x, typed), (g, _F32), (dout, typed),
        (entry_states, _F32), (out, typed), (dg, _F32), (workspace, _ANY))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _enqueue("kda_test_linear_scan_timeout", dev, stream, check, px, pg, pd, pe, T, H, d,
                    code, po, pdg, pw, wb, wait_ns)


def kda_linear_scan_step(x, g, state_in, state_out, h, N, H, d, dtype, stream=None,
                         check=True) -> int:
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (px, pg, pi, po, ph), dev = _args("kda_linear_scan_step", (x, typed), (g, _F32),
                                      (state_in, _F32), (state_out, _F32), (h, typed))
    return _enqueue("kda_linear_scan_step", dev, stream, check, px, pg, pi, po, ph, N, H, d, code)


def kda_fp8_pitch(K) -> int:
    return int(load().kda_fp8_pitch(K))


def kda_add_rms_norm(x, residual, w, rows, D, dtype, eps, sum, y, y8, y8_scale, stream=None,
                     check=True) -> int:
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (px, pr, pw, ps, py, p8, pc), dev = _args(
        "kda_add_rms_norm", (x, typed), (residual, typed), (w, _F32), (sum, typed), (y, typed),
        (y8, _FP8), (y8_scale, _F32))
    return _enqueue("kda_add_rms_norm", dev, stream, check, px, pr, pw, rows, D, code, eps, ps,
                    py, p8, pc)


@functools.lru_cache(maxsize=256)
def kda_add_rms_norm_bwd_workspace_size(rows, D) -> int:
    return int(load().kda_add_rms_norm_bwd_workspace_size(rows, D))


def kda_add_rms_norm_bwd(s, w, dy, dsum, rows, D, dtype, eps, dx, dw, workspace,
                         workspace_bytes=None, stream=None, check=True) -> int:
    code = dtype_code(dtype)
    typed = (_TORCH_OF[code],)
    (ps, pw, pd, pa, px, pg, pk), dev = _args(
        "kda_add_rms_norm_bwd", (s, typed), (w, _F32), (dy, typed), (dsum, typed), (dx, typed),
        (dw, _F32), (workspace, _ANY))
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    return _enqueue("kda_add_rms_norm_bwd", dev, stream, check, ps, pw, pd, pa, rows, D, code,
                    eps, px, pg, pk, wb)


def kda_quantize_fp8(x, rows, cols, dtype, block_rows, transpose, y8, scale, stream=None,
                     check=True) -> int:
    code = dtype_code(dtype)
    (px, p8, pc), dev = _args("kda_quantize_fp8", (x, (_TORCH_OF[code],)), (y8, _FP8),
                              (scale, _F32))
    return _enqueue("kda_quantize_fp8", dev, stream, check, px, rows, cols, code, block_rows,
                    int(bool(transpose)), p8, pc)


def kda_fp8_matmul(a8, a_scale, b8, b_scale, M, N, K, b_block_rows, out_dtype, out, stream=None,
                   check=True) -> int:
    code = dtype_code(out_dtype)
    (pa, ps, pb, pt, po), dev = _args("kda_fp8_matmul", (a8, _FP8), (a_scale, _F32), (b8, _FP8),
                                      (b_scale, _F32), (out, (_TORCH_OF[code],)))
    return _enqueue("kda_fp8_matmul", dev, stream, check, pa, ps, pb, pt, M, N, K, b_block_rows,
                    code, po)


def kda_test_fp8_matmul_timeout(a8, a_scale, b8, b_scale, M, N, K, b_block_rows, out_dtype, out,
                                withheld_cta, withheld_block, stream=None, check=True) -> int:
    """The product with one block of one CTA never loaded and shorter waits: exercises
    the bounded-wait error path (NaN).  Testing only."""
    code = dtype_code(out_dtype)
    (pa, ps, pb, pt, po), dev = _args("kda_test_fp8_matmul_timeout", (a8, _FP8), (a_scale, _F32),
                                      (b8, _FP8), (b_scale, _F32), (out, (_TORCH_OF[code],)))
    return _enqueue("kda_test_fp8_matmul_timeout", dev, stream, check, pa, ps, pb, pt, M, N, K,
                    b_block_rows, code, po, withheld_cta, withheld_block)


def kda_test_fp8_matmul_plan(M, N, K, b_block_rows, sms=148) -> tuple:
    """(tile_rows, split) of the kernel that kda_fp8_matmul takes.  Testing only."""
    rows, split = ctypes.c_int(), ctypes.c_int()
    st = load().kda_test_fp8_matmul_plan(M, N, K, b_block_rows, sms, ctypes.byref(rows),
                                         ctypes.byref(split))
    _ret(st, "kda_test_fp8_matmul_plan", True)
    return rows.value, split.value


def kda_chunk_fwd_noalloc(q, k, v, g, beta, initial_state, cu_seqlens, B, T, num_seqs, H, dk,
                          dv, chunk, dtype, o, final_state, stream=None, check=True) -> int:
    """kda_chunk_fwd without a workspace: for callers that may not allocate
    device memory.  The library's own static scratch array is used instead;
    see include/kda.h for its size limit and sharing rules."""
    _check("kda_chunk_fwd_noalloc", dtype, typed=(q, k, v, o), f32=(g, beta, initial_state,
           final_state), i32=(cu_seqlens,))
    st = load().kda_chunk_fwd_noalloc(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(initial_state),
                                      _p(cu_seqlens), B, T, num_seqs, H, dk, dv, chunk,
                                      dtype_code(dtype), _p(o), _p(final_state),
                                      _stream(stream))
    return _ret(st, "kda_chunk_fwd_noalloc", check)


def kda_get_device_status(workspace, stream=None) -> int:
    _check("kda_get_device_status", None, raw=(workspace,))
    return int(load().kda_get_device_status(_p(workspace), _stream(stream)))


# ------------------------------------------------------- allocating wrappers

def alloc_workspace(total_tokens, num_seqs, H, dk, dv, chunk, dtype, device="cuda"):
    n = kda_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv, chunk, dtype)
    if n == 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_chunk_fwd_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk=64,
              output_final_state=True, workspace=None, stream=None):
    """KDA chunkwise forward.  q, k [B, T, H, dk] or [T_total, H, dk] (packed with
    cu_seqlens); v likewise with dv; g like q (fp32); beta [.., H] (fp32).
    Returns (o, final_state or None).  All tensors on the current CUDA device."""
    packed = q.dim() == 3
    if packed:
        total, H, dk = q.shape
        B, T = 1, total
        N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else 1
        if cu_seqlens is None:
            B, T = 1, total
    else:
        B, T, H, dk = q.shape
        total, N = B * T, B
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens needs packed [T_total, H, d] inputs")
    dv = v.shape[-1]
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    hN = (torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
          if output_final_state else None)
    if workspace is None:
        workspace = alloc_workspace(total, N, H, dk, dv, chunk, q.dtype, q.device)
    kda_chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens, B, T, N, H, dk, dv, chunk,
                  q.dtype, o, hN, workspace, stream=stream)
    return o, hN


def chunk_bwd(q, k, v, g, beta, dout, initial_state=None, dfinal_state=None, cu_seqlens=None,
              head_gate=False, workspace=None, stream=None):
    """Gradients of sum(o * dout) + sum(final_state * dfinal_state) for
    chunk_fwd's inputs: returns (dq, dk, dv, dg, dbeta, dinitial_state), fp32,
    shaped like the inputs (dinitial_state [N, H, dk, dv]).  head_gate=True:
    g and dg are [.., H] (Gated DeltaNet)."""
    packed = q.dim() == 3
    if packed:
        total, H, dk = q.shape
        B, T = 1, total
        N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else 1
    else:
        B, T, H, dk = q.shape
        total, N = B * T, B
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens needs packed [T_total, H, d] inputs")
    dv = v.shape[-1]
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty(q.shape, **f32)
    dk_ = torch.empty(k.shape, **f32)
    dv_ = torch.empty(v.shape, **f32)
    dg = torch.empty(g.shape, **f32)
    db = torch.empty(beta.shape, **f32)
    dh0 = torch.empty(N, H, dk, dv, **f32)
    size = (kda_gdn_chunk_bwd_workspace_size if head_gate else kda_chunk_bwd_workspace_size)(
        total, N, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    call = kda_gdn_chunk_bwd if head_gate else kda_chunk_bwd
    call(q, k, v, g, beta, initial_state, dout, dfinal_state, cu_seqlens, B, T, N, H, dk, dv,
         q.dtype, dq, dk_, dv_, dg, db, dh0, workspace, stream=stream)
    return dq, dk_, dv_, dg, db, dh0


class ChunkKDA(torch.autograd.Function):
    """Differentiable KDA prefill: forward = chunk_fwd, backward = chunk_bwd (which
    recomputes the forward's per-chunk quantities, so only the inputs are
    saved).  Gradients of q, k, v are returned in their dtype."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_state, cu_seqlens, head_gate):
        if head_gate:
            packed = q.dim() == 3
            H, dk = q.shape[-2], q.shape[-1]
            B, T = (1, q.shape[0]) if packed else (q.shape[0], q.shape[1])
            total = B * T
            N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
            dv = v.shape[-1]
            o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            hN = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
            ws = torch.empty(kda_gdn_chunk_fwd_workspace_size(total, N, H, dk, dv, 64, q.dtype),
                             dtype=torch.uint8, device=q.device)
            kda_gdn_chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens, B, T, N, H, dk, dv, 64,
                              q.dtype, o, hN, ws)
        else:
            o, hN = chunk_fwd(q, k, v, g, beta, initial_state, cu_seqlens=cu_seqlens, chunk=64)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.head_gate = head_gate
        return o, hN

    @staticmethod
    def backward(ctx, do, dhN):
        q, k, v, g, beta, h0, cu = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.to(v.dtype).contiguous()
        dhN = None if dhN is None else dhN.float().contiguous()
        dq, dk, dv, dg, db, dh0 = chunk_bwd(q, k, v, g, beta, do, h0, dhN, cu,
                                            head_gate=ctx.head_gate)
        return (dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), dg, db,
                dh0 if h0 is not None else None, None, None)


def chunk_kda(q, k, v, g, beta, initial_state=None, cu_seqlens=None, head_gate=False):
    """Differentiable prefill: (o, final_state); see ChunkKDA."""
    return ChunkKDA.apply(q, k, v, g, beta, initial_state, cu_seqlens, head_gate)


def decode_step(q, k, v, g, beta, state, o=None, stream=None):
    """One recurrent step.  q, k, g [N, H, dk]; v [N, H, dv]; beta [N, H];
    state [N, H, dk, dv] fp32, updated in place.  Returns o [N, H, dv]."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(N, H, dv, dtype=v.dtype, device=v.device)
    kda_decode_step(q, k, v, g, beta, state, o, N, H, dk, dv, q.dtype, stream=stream)
    return o


# ----------------------------------------------------- gated linear recurrence

def _scan_shape(what, x, cu_seqlens):
    """(B, T, N, H, d) of x [B, T, H, d] or [T_total, H, d]."""
    if x.dim() == 3:
        total, H, d = x.shape
        return 1, total, 1 if cu_seqlens is None else cu_seqlens.numel() - 1, H, d
    if x.dim() != 4:
        raise ValueError(f"{what}: x is [B, T, H, d] or [T_total, H, d], got {tuple(x.shape)}")
    if cu_seqlens is not None:
        raise ValueError(f"{what}: cu_seqlens needs packed [T_total, H, d] inputs")
    B, T, H, d = x.shape
    return B, T, B, H, d


def _same_shape(what, shape, *named):
    """Each of the (name, tensor or None) pairs has the given shape."""
    for name, t in named:
        if t is not None and t.shape != shape:
            raise ValueError(f"{what}: {name} is {tuple(t.shape)}, expected {tuple(shape)}")


def linear_scan(x, g, initial_state=None, cu_seqlens=None, output_final_state=True,
                output_entry_states=False, workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel.  x [B, T,
    H, d] or [T_total, H, d] (packed with cu_seqlens), bf16 or fp32; g like x,
    fp32; initial_state [N, H, d] fp32.  Returns (h, final_state or None), and
    the entry states linear_scan_bwd takes if output_entry_states."""
    B, T, N, H, d = _scan_shape("linear_scan", x, cu_seqlens)
    _same_shape("linear_scan", x.shape, ("g", g))
    _same_shape("linear_scan", (N, H, d), ("initial_state", initial_state))
    total, f32 = B * T, dict(dtype=torch.float32, device=x.device)
    h = torch.empty_like(x)
    hN = torch.empty(N, H, d, **f32) if output_final_state else None
    entry = (torch.empty(kda_linear_scan_num_entries(total), H, d, **f32)
             if output_entry_states else None)
    if workspace is None:
        workspace = torch.empty(kda_linear_scan_workspace_size(total, H, d), dtype=torch.uint8,
                                device=x.device)
    kda_linear_scan_fwd(x, g, initial_state, cu_seqlens, B, T, N, H, d, x.dtype, h, hN, entry,
                        workspace, stream=stream)
    _used_on(stream, h, hN, entry, workspace)
    return (h, hN, entry) if output_entry_states else (h, hN)


def linear_scan_bwd(x, g, dout, initial_state=None, dfinal_state=None, cu_seqlens=None,
                    entry_states=None, workspace=None, stream=None):
    """Gradients of sum(h * dout) + sum(final_state * dfinal_state) for
    linear_scan's inputs: (dx like x, dg fp32, dinitial_state [N, H, d] fp32)."""
    B, T, N, H, d = _scan_shape("linear_scan_bwd", x, cu_seqlens)
    total, f32 = B * T, dict(dtype=torch.float32, device=x.device)
    _same_shape("linear_scan_bwd", x.shape, ("g", g), ("dout", dout))
    _same_shape("linear_scan_bwd", (N, H, d), ("initial_state", initial_state),
                ("dfinal_state", dfinal_state))
    _same_shape("linear_scan_bwd", (kda_linear_scan_num_entries(total), H, d),
                ("entry_states", entry_states))
    dx, dg = torch.empty_like(x), torch.empty(x.shape, **f32)
    dh0 = torch.empty(N, H, d, **f32)
    if workspace is None:
        workspace = torch.empty(kda_linear_scan_bwd_workspace_size(total, H, d),
                                dtype=torch.uint8, device=x.device)
    kda_linear_scan_bwd(x, g, initial_state, dout, dfinal_state, entry_states, cu_seqlens, B, T,
                        N, H, d, x.dtype, dx, dg, dh0, workspace, stream=stream)
    _used_on(stream, dx, dg, dh0, workspace)
    return dx, dg, dh0


def _check_leaves(ctx, device):
    """torch passes a leaf's gradient on on the stream that its accumulation node was
    made on, and that node lives as long as any graph of the leaf does.  The legacy
    default stream cannot join a capture: a backward pass captured while an eager
    graph from that stream lives would end the process, so the forward refuses."""
    stream = torch.cuda.current_stream(device).cuda_stream
    capturing = torch.cuda.is_current_stream_capturing()
    for node, _ in ctx.next_functions:
        if node is not None and hasattr(node, "variable"):
            if node.metadata.setdefault("kda_stream", stream) == 0 and capturing:
                raise RuntimeError("capturing a differentiable call while an eager graph of the "
                                   "same leaves, made on the default stream, is alive: release "
                                   "it (its outputs or loss) first")


class LinearScan(torch.autograd.Function):
    """Differentiable linear_scan; keeps its inputs and one state per 64 tokens."""

    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens):
        _check_leaves(ctx, x.device)
        ctx.set_materialize_grads(False)
        h, hN, entry = linear_scan(x, g, initial_state, cu_seqlens=cu_seqlens,
                                   output_entry_states=True)
        ctx.save_for_backward(x, g, initial_state, cu_seqlens, entry)
        return h, hN

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dhN):
        x, g, h0, cu, entry = ctx.saved_tensors
        dh = torch.zeros_like(x) if dh is None else dh.to(x.dtype).contiguous()
        dhN = None if dhN is None else dhN.float().contiguous()
        dx, dg, dh0 = linear_scan_bwd(x, g, dh, h0, dhN, cu_seqlens=cu, entry_states=entry)
        return dx, dg, dh0 if h0 is not None else None, None


def gated_linear_scan(x, g, initial_state=None, cu_seqlens=None):
    """Differentiable gated linear recurrence: (h, final_state); see LinearScan."""
    return LinearScan.apply(x, g, initial_state, cu_seqlens)


def linear_scan_step(x, g, state, h=None, state_out=None, stream=None):
    """One token of the recurrence.  x, g [N, H, d]; state [N, H, d] fp32, updated
    in place (or left alone, with the new one in state_out).  Returns h."""
    N, H, d = x.shape
    _same_shape("linear_scan_step", x.shape, ("g", g), ("state", state), ("h", h),
                ("state_out", state_out))
    made = h is None
    if made:
        h = torch.empty_like(x)
    kda_linear_scan_step(x, g, state, state if state_out is None else state_out, h, N, H, d,
                         x.dtype, stream=stream)
    if made:
        _used_on(stream, h)
    return h


# ----------------------------------- pre-norm, 8-bit matrices and their product

def _blocks128(n) -> int:
    return (n + 127) // 128


def _pitch(K) -> int:   # kda_fp8_pitch
    return (K + 15) // 16 * 16


def add_rms_norm(x, w, residual=None, eps=1e-6, quantize=False, sum=None, stream=None):
    """RMS norm of s = x + residual over the last dimension, times w (fp32).
    Returns (s, y), or with quantize=True (s, y8, scale): y as an 8-bit matrix
    (see quantize_fp8).  s is x itself without a residual; `sum` may be given for
    it (x or residual, to update it in place)."""
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _same_shape("add_rms_norm", x.shape, ("residual", residual), ("sum", sum))
    _same_shape("add_rms_norm", (D,), ("w", w))
    s = sum
    if s is None:
        s = x if residual is None else torch.empty_like(x)
    y = y8 = scale = None
    if quantize:
        y8 = torch.empty(rows, _pitch(D), dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(_blocks128(D), rows, dtype=torch.float32, device=x.device)
    else:
        y = torch.empty_like(x)
    kda_add_rms_norm(x, residual, w, rows, D, x.dtype, eps,
                     None if s is x and residual is None else s, y, y8, scale, stream=stream)
    _used_on(stream, s, y, y8, scale)
    return (s, y8, scale) if quantize else (s, y)


def add_rms_norm_bwd(s, w, dy, dsum=None, eps=1e-6, workspace=None, stream=None):
    """Gradients of sum(y * dy) + sum(s * dsum) for add_rms_norm: (dx, dw); dx is
    the gradient of x and of the residual."""
    D = s.shape[-1]
    rows = s.numel() // D if D else 0
    _same_shape("add_rms_norm_bwd", s.shape, ("dy", dy), ("dsum", dsum))
    _same_shape("add_rms_norm_bwd", (D,), ("w", w))
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    if workspace is None:
        workspace = torch.empty(kda_add_rms_norm_bwd_workspace_size(rows, D), dtype=torch.uint8,
                                device=s.device)
    kda_add_rms_norm_bwd(s, w, dy, dsum, rows, D, s.dtype, eps, dx, dw, workspace, stream=stream)
    _used_on(stream, dx, dw, workspace)
    return dx, dw


class AddRMSNorm(torch.autograd.Function):
    """Differentiable add_rms_norm: (s, y)."""

    @staticmethod
    def forward(ctx, x, w, residual, eps):
        _check_leaves(ctx, x.device)
        ctx.set_materialize_grads(False)
        s, y = add_rms_norm(x, w, residual, eps=eps)
        ctx.eps, ctx.has_residual = eps, residual is not None
        ctx.save_for_backward(s, w)
        return (s, y) if residual is not None else (s.view_as(s), y)

    @staticmethod
    @once_differentiable
    def backward(ctx, ds, dy):
        s, w = ctx.saved_tensors
        if dy is None:
            return ds, None, ds if ctx.has_residual else None, None
        ds = None if ds is None else ds.to(s.dtype).contiguous()
        dx, dw = add_rms_norm_bwd(s, w, dy.to(s.dtype).contiguous(), ds, eps=ctx.eps)
        return dx, dw, dx if ctx.has_residual else None, None


def residual_rms_norm(x, w, residual=None, eps=1e-6):
    """Differentiable residual addition and RMS norm: (x + residual, y)."""
    return AddRMSNorm.apply(x, w, residual, eps)


def quantize_fp8(x, block_rows=1, transpose=False, stream=None):
    """x [rows, cols] (bf16 or fp32) as an 8-bit matrix [R, K], x or its transpose:
    (y8, scale) with y8 [R, K rounded up to 16] float8_e4m3fn and scale [ceil(K /
    128), R] fp32, or [ceil(K / 128), ceil(R / 128)] with block_rows=128."""
    if x.dim() != 2:
        raise ValueError(f"quantize_fp8: x is [rows, cols], got {tuple(x.shape)}")
    rows, cols = x.shape
    R, K = (cols, rows) if transpose else (rows, cols)
    y8 = torch.empty(R, _pitch(K), dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(_blocks128(K), R if block_rows == 1 else _blocks128(R),
                        dtype=torch.float32, device=x.device)
    kda_quantize_fp8(x, rows, cols, x.dtype, block_rows, transpose, y8, scale, stream=stream)
    _used_on(stream, y8, scale)
    return y8, scale


def fp8_matmul(a8, a_scale, b8, b_scale, K=None, b_block_rows=128, out_dtype=torch.bfloat16,
               out=None, stream=None):
    """out [M, N] = a b^T of two 8-bit matrices as quantize_fp8 makes them, a with a
    scale per row, b per row (b_block_rows=1) or per 128 rows.  K: the number of
    columns that count, where the rows are padded."""
    M, N = a8.shape[0], b8.shape[0]
    if K is None:
        K = a8.shape[1]
    pitch, KB = _pitch(K), _blocks128(K)
    _same_shape("fp8_matmul", (M, pitch), ("a8", a8))
    _same_shape("fp8_matmul", (N, pitch), ("b8", b8))
    _same_shape("fp8_matmul", (KB, M), ("a_scale", a_scale))
    _same_shape("fp8_matmul", (KB, N if b_block_rows == 1 else _blocks128(N)),
                ("b_scale", b_scale))
    made = out is None
    if made:
        out = torch.empty(M, N, dtype=out_dtype, device=a8.device)
    else:
        _same_shape("fp8_matmul", (M, N), ("out", out))
    kda_fp8_matmul(a8, a_scale, b8, b_scale, M, N, K, b_block_rows, out.dtype, out, stream=stream)
    if made:
        _used_on(stream, out)
    return out


class Fp8Linear(torch.autograd.Function):
    """y = x w^T with both operands in 8 bits, forward and backward: x and the
    gradient of y with a scale per row and 128 columns (per column and 128 tokens
    for the weight's gradient), w with one per 128 x 128 block."""

    @staticmethod
    def forward(ctx, x, w):
        if w.dim() != 2 or x.shape[-1] != w.shape[1]:
            raise ValueError(f"fp8_linear: x {tuple(x.shape)} and w {tuple(w.shape)}")
        _check_leaves(ctx, x.device)
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        w8, w_scale = quantize_fp8(w, block_rows=128)
        x8, x_scale = quantize_fp8(x2)
        ctx.save_for_backward(x2, w)
        ctx.shape = x.shape
        y = fp8_matmul(x8, x_scale, w8, w_scale, K=w.shape[1], out_dtype=x.dtype)
        return y.view(*x.shape[:-1], w.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, w = ctx.saved_tensors
        (M, K), N = x2.shape, w.shape[0]
        dy2 = dy.reshape(M, N).to(x2.dtype).contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            d8, d_scale = quantize_fp8(dy2)
            wt8, wt_scale = quantize_fp8(w, block_rows=128, transpose=True)
            dx = fp8_matmul(d8, d_scale, wt8, wt_scale, K=N, out_dtype=x2.dtype).view(ctx.shape)
        if ctx.needs_input_grad[1]:
            if M == 0:
                return dx, torch.zeros_like(w)
            d8, d_scale = quantize_fp8(dy2, transpose=True)
            x8, x_scale = quantize_fp8(x2, transpose=True)
            dw = fp8_matmul(d8, d_scale, x8, x_scale, K=M, b_block_rows=1, out_dtype=w.dtype)
        return dx, dw


def fp8_linear(x, w):
    """Differentiable projection x [..., in] (bf16 or fp32) by w [out, in] with 8-bit
    operands; see Fp8Linear."""
    return Fp8Linear.apply(x, w)
