"""ctypes binding of libkda's C ABI (include/kda.h): argument marshalling only.

Every function below has the name of the C entry point it calls, takes torch
tensors (device memory) and plain numbers, and passes their pointers, sizes
and the current CUDA stream through unchanged.  No computation happens here;
if libkda.so is missing or fails to load, every call raises.
"""
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
# the same sources built with device-side bounds checks (KDA_DEBUG_CHECKS)
DEBUG_LIB_PATH = os.path.join(_HERE, "libkda_debug.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_MISALIGNED = 3
KDA_ERR_WORKSPACE = 4
KDA_ERR_CUDA = 5
KDA_ERR_TIMEOUT = 6
KDA_ERR_BAD_SEQLENS = 7
KDA_ERR_BOUNDS = 8

KDA_F32 = 0
KDA_BF16 = 1

KDA_ACT_NONE = 0
KDA_ACT_SILU = 1
KDA_NORM_RMS = 0
KDA_NORM_L2 = 1
KDA_ROT_HALVES = 0
KDA_ROT_PAIRS = 1

_VP = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "kda_status_string": (ctypes.c_char_p, [_I]),
    "kda_last_cuda_error_string": (ctypes.c_char_p, []),
    "kda_gate_fwd": (_I, [_VP, _VP, _F, _VP, _I64, _I, _I, _VP]),
    "kda_gate_bwd_workspace_size": (_SZ, [_I]),
    "kda_gate_bwd": (_I, [_VP, _VP, _F, _VP, _VP, _VP, _I64, _I, _I, _VP, _SZ, _VP]),
    "kda_chunk_fwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "kda_chunk_fwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I,
                           _F, _I, _VP, _VP, _VP, _SZ, _VP]),
    "kda_chunk_segment_transition": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _I, _I, _I, _I, _I,
                                          _I, _VP, _VP, _SZ, _VP]),
    "kda_chunk_state_prefix": (_I, [_VP, _I, _I, _VP, _I, _I, _I, _I, _VP, _VP]),
    "kda_chunk_fwd_gated": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _I, _VP, _VP, _I, _I, _I, _I,
                                 _I, _I, _F, _I, _VP, _VP, _VP, _SZ, _VP]),
    "kda_decode_step": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _VP, _I, _I, _I, _I, _F, _VP, _VP]),
    "kda_decode_step_gated": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _I, _VP, _I, _I, _I, _I, _F,
                                   _VP, _VP]),
    "kda_chunk_fwd_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                   _F, _I, _VP, _VP, _VP]),
    "kda_decode_verify": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _I, _VP, _I, _I, _I, _I, _I, _F,
                               _VP, _VP]),
    "kda_decode_replay": (_I, [_VP, _VP, _VP, _VP, _F, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I,
                               _VP]),
    "kda_chunk_fwd_gated_host_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "kda_chunk_fwd_gated_host": (_I, [_VP, _VP, _VP, _VP, _VP, _F, _VP, _I, _VP, _I, _I, _I, _I,
                                      _I, _F, _VP, _VP, _VP, _SZ, _VP, _VP]),
    "kda_recurrent_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "kda_recurrent_bwd": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                               _I, _I, _F, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "kda_short_conv_fwd": (_I, [_VP, _I64, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP,
                                _VP, _VP, _SZ, _VP]),
    "kda_short_conv_step": (_I, [_VP, _I64, _VP, _VP, _I, _VP, _I, _I, _I, _I, _VP, _VP]),
    "kda_short_conv_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "kda_short_conv_bwd": (_I, [_VP, _I64, _VP, _VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "kda_selective_scan_fwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "kda_selective_scan_fwd": (_I, [_VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP, _I64, _VP, _VP,
                                    _I64, _VP, _I, _I, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP,
                                    _VP, _VP, _SZ, _VP]),
    "kda_selective_scan_step": (_I, [_VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP, _I64, _VP, _VP,
                                     _I64, _VP, _I, _I, _VP, _I, _I, _I, _I, _VP, _VP]),
    "kda_selective_scan_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "kda_selective_scan_bwd": (_I, [_VP, _I64, _VP, _I64, _VP, _VP, _I64, _VP, _I64, _VP, _VP,
                                    _I64, _VP, _I, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                    _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                                    _VP]),
    "kda_qk_norm_fwd": (_I, [_VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                             _I, _I, _F, _VP, _VP, _VP]),
    "kda_qk_norm_bwd_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "kda_qk_norm_bwd": (_I, [_VP, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                             _I, _I, _F, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "kda_get_device_status": (_I, [_VP, _VP, ctypes.POINTER(ctypes.c_int32)]),
    "kda_noalloc_get_device_status": (_I, [ctypes.POINTER(ctypes.c_int32), _VP]),
    "kda_selftest_bounded_wait": (_I, [_VP, _I64, _VP]),
    "kda_debug_checks_enabled": (_I, []),
    "kda_selftest_bounds_check": (_I, [_VP, _VP]),
    "kda_set_wait_limit_ns": (_I, [_I64]),
}

_lib = None
_lib_path = LIB_PATH


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where} failed: {kda_status_string(status)} ({status})"
        if status == KDA_ERR_CUDA:
            msg += f" [{kda_last_cuda_error_string()}]"
        super().__init__(msg)


def _load(path):
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} not found at {path}; build it with "
            "`python -m gated_delta_rule_158_b200.build`")
    L = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib():
    """The selected library, libkda.so unless select_library(debug=True) was
    called (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def select_library(debug: bool):
    """Routes every call of this module to libkda_debug.so (debug=True) or
    libkda.so.  Returns the previously selected library's path."""
    global _lib, _lib_path
    prev = _lib_path
    path = DEBUG_LIB_PATH if debug else LIB_PATH
    if path != _lib_path or _lib is None:
        _lib = _load(path)
        _lib_path = path
    return prev


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("libkda takes contiguous tensors")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: building a Stream object costs 3 us a call.  The
        # function is looked up here, since a CPU-only torch has none and the
        # package's host side works there
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _check(status, where):
    if status != KDA_OK:
        raise KdaError(status, where)


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def kda_last_cuda_error_string() -> str:
    return lib().kda_last_cuda_error_string().decode()


def kda_gate_fwd(z, A_log, g, g_min=-5.0, stream=None):
    """g = g_min * sigmoid(exp(A_log[h]) * z); z, g fp32 [..., H, dk]."""
    H, dk = z.shape[-2], z.shape[-1]
    rows = z.numel() // (H * dk) if z.numel() else 0
    _check(lib().kda_gate_fwd(_ptr(z), _ptr(A_log), float(g_min), _ptr(g), rows, H, dk,
                              _stream(stream)), "kda_gate_fwd")


def kda_gate_bwd_workspace_size(H) -> int:
    return int(lib().kda_gate_bwd_workspace_size(H))


def kda_gate_bwd(z, A_log, dg, dz, dA_log, workspace, g_min=-5.0, stream=None):
    """dz [..., H, dk] and dA_log [H] from dg through the gate
    g = g_min * sigmoid(exp(A_log[h]) * z); dz may be dg itself."""
    H, dk = z.shape[-2], z.shape[-1]
    rows = z.numel() // (H * dk) if z.numel() else 0
    _check(lib().kda_gate_bwd(_ptr(z), _ptr(A_log), float(g_min), _ptr(dg), _ptr(dz),
                              _ptr(dA_log), rows, H, dk, _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "kda_gate_bwd")


def kda_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs=0, chunk_size=0,
                                 in_dtype=KDA_BF16) -> int:
    return int(lib().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, chunk_size,
                                                  in_dtype))


def kda_chunk_fwd(q, k, v, g, beta, out, workspace, init_state=None, cu_seqlens=None,
                  final_state=None, scale=1.0, chunk_size=0, stream=None):
    """Chunkwise forward; q, k, g [B,T,H,dk], v/out [B,T,H,dv], beta [B,T,H]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(lib().kda_chunk_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dtype(q), _ptr(init_state),
        _ptr(cu_seqlens), num_seqs, B, T, H, dk, dv, float(scale), int(chunk_size), _ptr(out),
        _ptr(final_state), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "kda_chunk_fwd")


def kda_chunk_fwd_noalloc(q, k, v, g, beta, out, init_state=None, cu_seqlens=None,
                          final_state=None, scale=1.0, chunk_size=0, stream=None):
    """kda_chunk_fwd using the library's built-in scratch instead of a workspace,
    for callers that cannot allocate device memory (see include/kda.h)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(lib().kda_chunk_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dtype(q), _ptr(init_state),
        _ptr(cu_seqlens), num_seqs, B, T, H, dk, dv, float(scale), int(chunk_size), _ptr(out),
        _ptr(final_state), _stream(stream)), "kda_chunk_fwd_noalloc")


def kda_chunk_fwd_gated(q, k, v, z, A_log, beta, out, workspace, g_min=-5.0, init_state=None,
                        cu_seqlens=None, final_state=None, scale=1.0, chunk_size=0, stream=None):
    """kda_chunk_fwd with the gate fused in: z [B,T,H,dk] and A_log [H] replace g."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(lib().kda_chunk_fwd_gated(
        _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), float(g_min), _ptr(beta), _dtype(q),
        _ptr(init_state), _ptr(cu_seqlens), num_seqs, B, T, H, dk, dv, float(scale),
        int(chunk_size), _ptr(out), _ptr(final_state), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "kda_chunk_fwd_gated")


def kda_chunk_segment_transition(q, k, v, z, A_log, beta, pairs, workspace, g_min=-5.0,
                                 stream=None):
    """Per (b, h) of the segment given: pairs[b, h, 0] = S~ (from a zero state),
    pairs[b, h, 1] = M (the segment's transition); pairs fp32 [B, H, 2, 128, 128]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib().kda_chunk_segment_transition(
        _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), float(g_min), _ptr(beta), _dtype(q),
        B, T, H, dk, dv, _ptr(pairs), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "kda_chunk_segment_transition")


def kda_chunk_state_prefix(pairs, index, state_out, init_state=None, stream=None):
    """Incoming state of segment `index` from the pairs [count, B, H, 2, dk, dv] of the
    segments in order: S_in[0] = init (or 0), S_in[r + 1] = S~_r + M_r S_in[r]."""
    count, B, H = pairs.shape[0], pairs.shape[1], pairs.shape[2]
    dk, dv = pairs.shape[-2], pairs.shape[-1]
    _check(lib().kda_chunk_state_prefix(_ptr(pairs), count, int(index), _ptr(init_state), B, H,
                                        dk, dv, _ptr(state_out), _stream(stream)),
           "kda_chunk_state_prefix")


def kda_decode_step_gated(q, k, v, z, A_log, beta, state, out, g_min=-5.0, scale=1.0,
                          stream=None):
    """kda_decode_step with the gate fused in: z [N,H,dk] and A_log [H] replace g."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib().kda_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log),
                                       float(g_min), _ptr(beta), _dtype(q), _ptr(state), N, H,
                                       dk, dv, float(scale), _ptr(out), _stream(stream)),
           "kda_decode_step_gated")


def kda_decode_step(q, k, v, g, beta, state, out, scale=1.0, stream=None):
    """One decode step; q, k, g [N,H,dk], v/out [N,H,dv], beta [N,H], state in place."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dtype(q),
                                 _ptr(state), N, H, dk, dv, float(scale), _ptr(out),
                                 _stream(stream)), "kda_decode_step")


def kda_decode_verify(q, k, v, g, beta, state, out, A_log=None, g_min=-5.0, scale=1.0,
                      stream=None):
    """Outputs of K draft tokens per sequence, state read only.  q, k, g
    [N,K,H,dk], v/out [N,K,H,dv], beta [N,K,H]; g is z when A_log is given."""
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib().kda_decode_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(A_log),
                                   float(g_min), _ptr(beta), _dtype(q), _ptr(state), N, H, K, dk,
                                   dv, float(scale), _ptr(out), _stream(stream)),
           "kda_decode_verify")


def kda_decode_replay(k, v, g, beta, state, accept_len, A_log=None, g_min=-5.0, stream=None):
    """Apply each sequence's first accept_len[n] tokens to the state in place."""
    N, K, H, dk = k.shape
    dv = v.shape[-1]
    _check(lib().kda_decode_replay(_ptr(k), _ptr(v), _ptr(g), _ptr(A_log), float(g_min),
                                   _ptr(beta), _dtype(k), _ptr(state), _ptr(accept_len), N, H, K,
                                   dk, dv, _stream(stream)), "kda_decode_replay")


def kda_chunk_fwd_gated_host_workspace_size(B, T, H, dk, dv, in_dtype=KDA_BF16) -> int:
    return int(lib().kda_chunk_fwd_gated_host_workspace_size(B, T, H, dk, dv, in_dtype))


def kda_chunk_fwd_gated_host(q, k, v, z, A_log, beta, out, workspace, g_min=-5.0,
                             init_state=None, final_state=None, scale=1.0, stream=None,
                             copy_stream=None):
    """Gated chunked prefill of a dense batch in host memory (CPU tensors,
    page-locked for overlap): q, k [B,T,H,dk], v [B,T,H,dv], z [B,T,H,dk]
    fp32, A_log [H], beta [B,T,H]; out [B,T,H,dv] and final_state
    [B,H,dk,dv] are host tensors written by the time `stream` reaches the end
    of the call's work.  workspace is a device uint8 tensor."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, z, A_log, beta, out, init_state, final_state):
        if t is not None and t.is_cuda:
            raise ValueError("kda_chunk_fwd_gated_host takes host tensors")
    _check(lib().kda_chunk_fwd_gated_host(
        _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(A_log), float(g_min), _ptr(beta), _dtype(q),
        _ptr(init_state), B, T, H, dk, dv, float(scale), _ptr(out), _ptr(final_state),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        None if copy_stream is None else _stream(copy_stream)), "kda_chunk_fwd_gated_host")


def kda_recurrent_bwd_workspace_size(B, T, H, dk, dv, num_seqs=0) -> int:
    return int(lib().kda_recurrent_bwd_workspace_size(B, T, H, dk, dv, num_seqs))


def kda_recurrent_bwd(q, k, v, g, beta, dout, grads, workspace, init_state=None, d_final=None,
                      cu_seqlens=None, scale=1.0, stream=None):
    """Gradients through the recurrence.  q, k, g [B,T,H,dk]; v, dout
    [B,T,H,dv]; beta [B,T,H]; cu_seqlens (int32 [N+1], B == 1) for a packed
    batch.  `grads` is a dict of fp32 output tensors dq, dk, dg [B,T,H,dk],
    dv [B,T,H,dv], dbeta [B,T,H] and optionally d_init [N,H,dk,dv]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(lib().kda_recurrent_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dtype(q), _ptr(init_state), _ptr(dout),
        _ptr(d_final), _ptr(cu_seqlens), N, B, T, H, dk, dv, float(scale), _ptr(grads["dq"]),
        _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dg"]), _ptr(grads["dbeta"]),
        _ptr(grads.get("d_init")), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "kda_recurrent_bwd")


# ---- the operators around the recurrence: their inputs may be row slices of
# wider tensors, so shapes, types and devices are checked here.  A decode loop
# makes these calls once per layer and token, and the checks are most of a
# call's host time: they ask one question per tensor and explain a no later.

_F32T = torch.float32


def _arg(dev, name, t, shape, dtype):
    """The pointer of a dense CUDA tensor of this shape and type on device
    `dev`, the current one."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(dev, name, t, shape, dtype)
    raise ValueError(f"{name}: expected a dense tensor")


def _opt(dev, name, t, shape, dtype):
    return None if t is None else _arg(dev, name, t, shape, dtype)


def _refuse(dev, name, t, shape, dtype):
    """Raises what is wrong with the tensor, if it is not its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device")


_INT_MAX = 0x7FFFFFFF  # sizes a, b >= 0: a | b is above it where one of them is


def _too_large(*sizes):
    # ctypes would cut an int of more than 32 bits down without a word
    raise ValueError(f"sizes {sizes}: at most 2^31 - 1 each")


def _rows(dev, name, t, shape, lead, width, dtype):
    """(pointer, row stride) of a tensor whose first `lead` dimensions number
    its rows of `width` elements: rows dense, any constant distance apart."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if t.is_contiguous():
                return t.data_ptr(), width
        else:
            _refuse(dev, name, t, shape, dtype)
    except AttributeError:
        _refuse(dev, name, t, shape, dtype)
    strides, dense = t.stride(), 1
    for n, st in zip(reversed(shape[lead:]), reversed(strides[lead:])):
        if n > 1 and st != dense:
            raise ValueError(f"{name}: rows must be dense")
        dense *= n
    stride = None
    for n, st in zip(reversed(shape[:lead]), reversed(strides[:lead])):
        if n == 1:
            continue
        if stride is None:
            stride, reach = st, st * n
        elif st != reach:
            raise ValueError(f"{name}: rows must be a constant distance apart")
        else:
            reach *= n
    if stride is None:
        stride = width
    if stride < width:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), stride


def _grad(dev, grads, name, shape):
    return _arg(dev, f"grads['{name}']", grads.get(name), shape, _F32T)


def _opt_grad(dev, grads, name, shape):
    t = grads.get(name)
    return None if t is None else _arg(dev, f"grads['{name}']", t, shape, _F32T)


def _offsets(dev, cu_seqlens, batch):
    """(pointer, number of packed sequences, number of states)"""
    if cu_seqlens is None:
        return None, 0, batch
    n = cu_seqlens.numel() - 1
    if n > _INT_MAX:
        _too_large(n)
    return _arg(dev, "cu_seqlens", cu_seqlens, (n + 1,), torch.int32), n, n


def _scratch(dev, workspace):
    if workspace is None:
        return None, 0
    return (_arg(dev, "workspace", workspace, workspace.shape, workspace.dtype),
            workspace.numel() * workspace.element_size())


def _on(stream, dev):
    # as _stream, for a device that is known
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def kda_short_conv_fwd(x, weight, out, workspace, bias=None, init_state=None, cu_seqlens=None,
                       final_state=None, activation=KDA_ACT_SILU, stream=None):
    """Causal convolution of each channel over its sequence's tokens; x [B,T,D]
    (rows may be slices of a wider tensor), weight fp32 [D,W], out [B,T,D],
    states [N,W-1,D] of x's type."""
    dev = torch.cuda.current_device()
    shape, dt, code = x.shape, x.dtype, _dtype(x)
    B, T, D = shape
    W = weight.shape[-1]
    cu, num, N = _offsets(dev, cu_seqlens, B)
    if (B | T | D | W) > _INT_MAX:
        _too_large(B, T, D, W)
    xp, xs = _rows(dev, "x", x, shape, 2, D, dt)
    ws, wsb = _scratch(dev, workspace)
    _check(lib().kda_short_conv_fwd(
        xp, xs, _arg(dev, "weight", weight, (D, W), _F32T), _opt(dev, "bias", bias, (D,), _F32T),
        code, _opt(dev, "init_state", init_state, (N, W - 1, D), dt), cu, num, B, T, D, W,
        activation, _arg(dev, "out", out, shape, dt),
        _opt(dev, "final_state", final_state, (N, W - 1, D), dt), ws, wsb, _on(stream, dev)),
        "kda_short_conv_fwd")


def kda_short_conv_step(x, weight, state, out, bias=None, activation=KDA_ACT_SILU, stream=None):
    """One token of N sequences: x, out [N,D], state [N,W-1,D] shifted in place."""
    dev = torch.cuda.current_device()
    shape, dt, code = x.shape, x.dtype, _dtype(x)
    N, D = shape
    W = weight.shape[-1]
    if (N | D | W) > _INT_MAX:
        _too_large(N, D, W)
    xp, xs = _rows(dev, "x", x, shape, 1, D, dt)
    _check(lib().kda_short_conv_step(
        xp, xs, _arg(dev, "weight", weight, (D, W), _F32T), _opt(dev, "bias", bias, (D,), _F32T),
        code, _arg(dev, "state", state, (N, W - 1, D), dt), N, D, W, activation,
        _arg(dev, "out", out, shape, dt), _on(stream, dev)), "kda_short_conv_step")


def kda_short_conv_bwd_workspace_size(B, T, D, W, num_seqs=0) -> int:
    if (B | T | D | W | num_seqs) > _INT_MAX:
        _too_large(B, T, D, W, num_seqs)
    return int(lib().kda_short_conv_bwd_workspace_size(B, T, D, W, num_seqs))


def kda_short_conv_bwd(x, weight, dout, grads, workspace, bias=None, init_state=None,
                       d_final=None, cu_seqlens=None, activation=KDA_ACT_SILU, stream=None):
    """Gradients of kda_short_conv_fwd.  dout fp32 [B,T,D]; `grads` is a dict of
    fp32 outputs dx [B,T,D], dweight [D,W] and optionally dbias [D], d_init
    [N,W-1,D]."""
    dev = torch.cuda.current_device()
    shape, dt, code = x.shape, x.dtype, _dtype(x)
    B, T, D = shape
    W = weight.shape[-1]
    cu, num, N = _offsets(dev, cu_seqlens, B)
    if (B | T | D | W) > _INT_MAX:
        _too_large(B, T, D, W)
    xp, xs = _rows(dev, "x", x, shape, 2, D, dt)
    ws, wsb = _scratch(dev, workspace)
    _check(lib().kda_short_conv_bwd(
        xp, xs, _arg(dev, "weight", weight, (D, W), _F32T), _opt(dev, "bias", bias, (D,), _F32T),
        code, _opt(dev, "init_state", init_state, (N, W - 1, D), dt),
        _arg(dev, "dout", dout, shape, _F32T),
        _opt(dev, "d_final", d_final, (N, W - 1, D), _F32T), cu, num, B, T, D, W, activation,
        _grad(dev, grads, "dx", shape), _grad(dev, grads, "dweight", (D, W)),
        _opt_grad(dev, grads, "dbias", (D,)), _opt_grad(dev, grads, "d_init", (N, W - 1, D)), ws,
        wsb, _on(stream, dev)), "kda_short_conv_bwd")


def kda_selective_scan_fwd_workspace_size(B, T, D, S, G=1, num_seqs=0) -> int:
    if (B | T | D | S | G | num_seqs) > _INT_MAX:
        _too_large(B, T, D, S, G, num_seqs)
    return int(lib().kda_selective_scan_fwd_workspace_size(B, T, D, S, G, num_seqs))


def _scan_inputs(dev, n, x, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus):
    """The marshalled input arguments that the scan's entries share; x has `n`
    dimensions in front of its channels."""
    shape, dt, code = x.shape, x.dtype, _dtype(x)
    if len(shape) != n + 1:
        raise ValueError(f"x: shape {tuple(shape)}, expected {n + 1} dimensions")
    ch = shape[-1]
    (S,), (G,) = A.shape[-1:], Bm.shape[-2:-1]
    if max(*shape, S, G) > _INT_MAX:
        _too_large(*shape, S, G)
    mix, w = (*shape[:-1], G, S), G * S
    return (*_rows(dev, "x", x, shape, n, ch, dt), *_rows(dev, "delta", delta, shape, n, ch, dt),
            _arg(dev, "A", A, (ch, S), _F32T), *_rows(dev, "Bm", Bm, mix, n, w, dt),
            *_rows(dev, "Cm", Cm, mix, n, w, dt), _opt(dev, "D", D, (ch,), _F32T),
            *((None, 0) if z is None else _rows(dev, "z", z, shape, n, ch, dt)),
            _opt(dev, "delta_bias", delta_bias, (ch,), _F32T), 1 if delta_softplus else 0,
            code), ch, S, G


def kda_selective_scan_fwd(x, delta, A, Bm, Cm, out, workspace, D=None, z=None, delta_bias=None,
                           delta_softplus=True, init_state=None, cu_seqlens=None,
                           final_state=None, stream=None):
    """Selective state space scan; x, delta, z, out [B,T,D], Bm, Cm [B,T,G,S]
    (inputs may be row slices of wider tensors), A fp32 [D,S], D and delta_bias
    fp32 [D], states fp32 [N,D,S]."""
    dev = torch.cuda.current_device()
    args, ch, S, G = _scan_inputs(dev, 2, x, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus)
    B, T = x.shape[:2]
    cu, num, N = _offsets(dev, cu_seqlens, B)
    ws, wsb = _scratch(dev, workspace)
    _check(lib().kda_selective_scan_fwd(
        *args, _opt(dev, "init_state", init_state, (N, ch, S), _F32T), cu, num, B, T, ch, S, G,
        _arg(dev, "out", out, (B, T, ch), x.dtype),
        _opt(dev, "final_state", final_state, (N, ch, S), _F32T), ws, wsb, _on(stream, dev)),
        "kda_selective_scan_fwd")


def kda_selective_scan_step(x, delta, A, Bm, Cm, state, out, D=None, z=None, delta_bias=None,
                            delta_softplus=True, stream=None):
    """One token of N sequences: x, delta, z, out [N,D], Bm, Cm [N,G,S], state
    fp32 [N,D,S] in place."""
    dev = torch.cuda.current_device()
    args, ch, S, G = _scan_inputs(dev, 1, x, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus)
    N = x.shape[0]
    _check(lib().kda_selective_scan_step(
        *args, _arg(dev, "state", state, (N, ch, S), _F32T), N, ch, S, G,
        _arg(dev, "out", out, (N, ch), x.dtype), _on(stream, dev)), "kda_selective_scan_step")


def kda_selective_scan_bwd_workspace_size(B, T, D, S, G=1, num_seqs=0) -> int:
    if (B | T | D | S | G | num_seqs) > _INT_MAX:
        _too_large(B, T, D, S, G, num_seqs)
    return int(lib().kda_selective_scan_bwd_workspace_size(B, T, D, S, G, num_seqs))


def kda_selective_scan_bwd(x, delta, A, Bm, Cm, dout, grads, workspace, D=None, z=None,
                           delta_bias=None, delta_softplus=True, init_state=None, d_final=None,
                           cu_seqlens=None, stream=None):
    """Gradients of kda_selective_scan_fwd.  dout has x's type; `grads` is a
    dict of fp32 outputs dx, ddelta [B,T,D], dA [D,S], dB, dC [B,T,G,S], dz
    [B,T,D] with z, and optionally dD, ddelta_bias [D], d_init [N,D,S]."""
    dev = torch.cuda.current_device()
    args, ch, S, G = _scan_inputs(dev, 2, x, delta, A, Bm, Cm, D, z, delta_bias, delta_softplus)
    B, T = x.shape[:2]
    cu, num, N = _offsets(dev, cu_seqlens, B)
    ws, wsb = _scratch(dev, workspace)
    rows, mix, state = (B, T, ch), (B, T, G, S), (N, ch, S)
    _check(lib().kda_selective_scan_bwd(
        *args, _opt(dev, "init_state", init_state, state, _F32T),
        _arg(dev, "dout", dout, rows, x.dtype), _opt(dev, "d_final", d_final, state, _F32T), cu,
        num, B, T, ch, S, G, _grad(dev, grads, "dx", rows), _grad(dev, grads, "ddelta", rows),
        _grad(dev, grads, "dA", (ch, S)), _grad(dev, grads, "dB", mix),
        _grad(dev, grads, "dC", mix), _opt_grad(dev, grads, "dD", (ch,)),
        _opt_grad(dev, grads, "dz", rows), _opt_grad(dev, grads, "ddelta_bias", (ch,)),
        _opt_grad(dev, grads, "d_init", state), ws, wsb, _on(stream, dev)),
        "kda_selective_scan_bwd")


def _norm_inputs(dev, q, k, q_weight, k_weight, positions, inv_freq, mode, rotation, eps):
    """The marshalled input arguments that the norms' entries share, and the
    shapes of q and k."""
    shape, dt, code = q.shape, q.dtype, _dtype(q)
    *lead, Hq, dim = shape
    Hk = k.shape[-2]
    k_shape, n, tokens = (*lead, Hk, dim), len(lead), math.prod(lead)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if (tokens | Hq | Hk | dim | rot) > _INT_MAX:
        _too_large(tokens, Hq, Hk, dim, rot)
    return (*_rows(dev, "q", q, shape, n, Hq * dim, dt),
            *_rows(dev, "k", k, k_shape, n, Hk * dim, dt),
            _opt(dev, "q_weight", q_weight, (dim,), _F32T),
            _opt(dev, "k_weight", k_weight, (dim,), _F32T),
            _opt(dev, "positions", positions, shape[:-2], torch.int32),
            _opt(dev, "inv_freq", inv_freq, (rot // 2,), _F32T), code, tokens, Hq, Hk, dim, rot,
            mode, rotation, eps), shape, k_shape


def kda_qk_norm_fwd(q, k, q_out, k_out, q_weight=None, k_weight=None, positions=None,
                    inv_freq=None, mode=KDA_NORM_L2, rotation=KDA_ROT_HALVES, eps=1e-6,
                    stream=None):
    """Norm of every head's query and key row, then the rotation of its first
    2 * inv_freq.numel() elements by positions [...] (int32) times inv_freq
    (fp32).  q [..., Hq, d], k [..., Hk, d] (rows of a token may be slices of
    a wider tensor); q_out, k_out dense, of the same type, or q, k themselves."""
    dev = torch.cuda.current_device()
    args, qs, ks = _norm_inputs(dev, q, k, q_weight, k_weight, positions, inv_freq, mode,
                                rotation, eps)
    _check(lib().kda_qk_norm_fwd(
        *args, _arg(dev, "q_out", q_out, qs, q.dtype), _arg(dev, "k_out", k_out, ks, q.dtype),
        _on(stream, dev)), "kda_qk_norm_fwd")


def kda_qk_norm_bwd_workspace_size(tokens, Hq, Hk, d) -> int:
    if (tokens | Hq | Hk | d) > _INT_MAX:
        _too_large(tokens, Hq, Hk, d)
    return int(lib().kda_qk_norm_bwd_workspace_size(tokens, Hq, Hk, d))


def kda_qk_norm_bwd(q, k, dq_out, dk_out, grads, workspace=None, q_weight=None, k_weight=None,
                    positions=None, inv_freq=None, mode=KDA_NORM_L2, rotation=KDA_ROT_HALVES,
                    eps=1e-6, stream=None):
    """Gradients of kda_qk_norm_fwd.  dq_out, dk_out fp32; `grads` is a dict of
    fp32 outputs dq, dk (dq may be dq_out itself, dk dk_out) and optionally
    dq_weight, dk_weight [d], which need the workspace."""
    dev = torch.cuda.current_device()
    args, qs, ks = _norm_inputs(dev, q, k, q_weight, k_weight, positions, inv_freq, mode,
                                rotation, eps)
    dim = qs[-1]
    ws, wsb = _scratch(dev, workspace)
    _check(lib().kda_qk_norm_bwd(
        *args, _arg(dev, "dq_out", dq_out, qs, _F32T), _arg(dev, "dk_out", dk_out, ks, _F32T),
        _grad(dev, grads, "dq", qs), _grad(dev, grads, "dk", ks),
        _opt_grad(dev, grads, "dq_weight", (dim,)), _opt_grad(dev, grads, "dk_weight", (dim,)),
        ws, wsb, _on(stream, dev)), "kda_qk_norm_bwd")


def kda_get_device_status(workspace, stream=None):
    """(status, detail) recorded on the device in this workspace; syncs the stream."""
    detail = ctypes.c_int32(0)
    st = lib().kda_get_device_status(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def kda_noalloc_get_device_status(stream=None):
    """(status, detail) that the last kda_chunk_fwd_noalloc call on the current
    device recorded in the library's built-in scratch; syncs the stream."""
    detail = ctypes.c_int32(0)
    st = lib().kda_noalloc_get_device_status(ctypes.byref(detail), _stream(stream))
    return int(st), int(detail.value)


def kda_set_wait_limit_ns(limit_ns):
    """Diagnostic: bound of the chunk kernel's internal waits (default 2e9 ns)."""
    _check(lib().kda_set_wait_limit_ns(int(limit_ns)), "kda_set_wait_limit_ns")


def kda_debug_checks_enabled() -> bool:
    return bool(lib().kda_debug_checks_enabled())


def kda_selftest_bounds_check(workspace, stream=None):
    _check(lib().kda_selftest_bounds_check(_ptr(workspace), _stream(stream)),
           "kda_selftest_bounds_check")


def kda_selftest_bounded_wait(workspace, spin_limit_ns, stream=None):
    _check(lib().kda_selftest_bounded_wait(_ptr(workspace), int(spin_limit_ns),
                                           _stream(stream)), "kda_selftest_bounded_wait")
