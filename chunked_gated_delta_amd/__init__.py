"""Python binding of libkda.so, the MI355X KDA chunked forward library.

Argument marshalling only: every step of the forward pass runs in the HIP
kernels behind the C ABI of include/kda.h.  The names mirror that header:
``kda_fwd``, ``kda_workspace_size``, ``kda_is_supported``, ``kda_shard_affine``,
``kda_shard_scan``, ``kda_decode``, ``kda_fwd_ex`` (with the ``FLAG_*`` variant bits),
``kda_bwd``, ``kda_bwd_ex``, ``kda_bwd_workspace_size``,
``kda_workspace_faults`` (with the ``FAULT_*`` bits), ``kda_fwd_noalloc`` and the operators around
the core: the gated linear recurrence (``kda_glr_fwd``, ``kda_glr_bwd``, ``kda_glr_step``), the short
causal convolution (``kda_conv_fwd``, ``kda_conv_bwd``, ``kda_conv_step``) and the norm and rotation
of queries and keys (``kda_qk_rope_fwd``, ``kda_qk_rope_bwd``), and the token mixers beside the
core: linear attention with a decay for each head (``kda_la_fwd``, ``kda_la_bwd``, ``kda_la_step``) and
causal softmax attention (``kda_attn_fwd``, ``kda_attn_bwd``).  PyTorch provides
device memory and the current stream; there is no CPU or PyTorch fallback, and
importing this module fails if the library has not been built.
"""

from __future__ import annotations

import ctypes
import math
import os

# torch first: its bundled HIP runtime carries the same SONAME
# (libamdhip64.so.7) that libkda.so links against, so loading torch first makes
# both use one runtime.  Loading libkda.so first would put a second HIP runtime
# in the process, and whichever initialises second sees no device.
import torch  # noqa: F401

__all__ = ["kda_fwd", "kda_fwd_ex", "kda_workspace_size", "kda_is_supported", "kda_shard_affine",
           "kda_shard_scan", "kda_decode", "kda_bwd", "kda_bwd_ex", "kda_bwd_workspace_size",
           "kda_workspace_faults", "kda_fwd_noalloc", "NOALLOC_SCRATCH_BYTES", "FAULT_WAIT_TIMEOUT", "FAULT_GATE_RANGE", "FAULT_QK_NORM", "KdaError", "STATUS", "library_path", "exported_symbols",
           "FLAG_GATE_GIVEN", "FLAG_BETA_GIVEN", "FLAG_NO_QK_NORM", "FLAG_STATE_VK", "FLAG_REUSE_RECORDS",
           "FLAG_KEEP_RECORDS", "FLAG_SINGLE_LAUNCH", "FAULT_PLACEMENT", "FLAG_COMPLEMENT", "FLAG_SILU",
           "FLAG_RMS_NORM", "FLAG_INTERLEAVED", "FLAG_ZERO_REST", "kda_glr_fwd", "kda_glr_bwd", "kda_glr_step",
           "kda_glr_workspace_size", "kda_glr_states_size", "kda_glr_bwd_workspace_size", "kda_conv_fwd",
           "kda_conv_bwd", "kda_conv_step", "kda_conv_bwd_workspace_size", "kda_qk_rope_fwd", "kda_qk_rope_bwd",
           "kda_qk_rope_bwd_workspace_size", "kda_la_fwd", "kda_la_bwd", "kda_la_step", "kda_la_workspace_size",
           "kda_la_bwd_workspace_size", "kda_attn_fwd", "kda_attn_bwd", "kda_attn_workspace_size",
           "kda_attn_bwd_workspace_size"]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libkda.so")

STATUS = {0: "KDA_SUCCESS", 1: "KDA_ERR_INVALID", 2: "KDA_ERR_UNSUPPORTED",
          3: "KDA_ERR_WORKSPACE", 4: "KDA_ERR_LAUNCH"}
exported_symbols = ("kda_fwd", "kda_workspace_size", "kda_is_supported", "kda_status_string",
                    "kda_shard_affine", "kda_shard_scan", "kda_decode", "kda_fwd_ex", "kda_bwd",
                    "kda_bwd_ex", "kda_bwd_workspace_size", "kda_workspace_faults", "kda_fwd_noalloc",
                    "kda_glr_fwd", "kda_glr_bwd", "kda_glr_step", "kda_glr_workspace_size", "kda_glr_states_size",
                    "kda_glr_bwd_workspace_size", "kda_conv_fwd", "kda_conv_bwd", "kda_conv_step",
                    "kda_conv_bwd_workspace_size", "kda_qk_rope_fwd", "kda_qk_rope_bwd",
                    "kda_qk_rope_bwd_workspace_size", "kda_la_fwd", "kda_la_bwd", "kda_la_step",
                    "kda_la_workspace_size", "kda_la_bwd_workspace_size", "kda_attn_fwd", "kda_attn_bwd",
                    "kda_attn_workspace_size", "kda_attn_bwd_workspace_size")
# kda_fwd_ex variant bits (KDA_FLAG_* in include/kda.h)
FLAG_GATE_GIVEN, FLAG_BETA_GIVEN, FLAG_NO_QK_NORM, FLAG_STATE_VK = 1, 2, 4, 8
# kda_fwd_ex, kda_bwd_ex: reuse the chunk records the previous call left in the workspace
FLAG_REUSE_RECORDS = 16
# kda_fwd_ex: leave every chunk record in the workspace, for a later FLAG_REUSE_RECORDS call
FLAG_KEEP_RECORDS = 32
# kda_fwd_ex: one-sequence calls with >= 16 heads run as one producer/chain launch
FLAG_SINGLE_LAUNCH = 64
# variant bits of the operators around the core: recurrence input scaled by 1 - a; convolution
# followed by SiLU; q, k divided by their root mean square; rotated pairs (2i, 2i + 1); rows
# behind the last sequence written as zeros
FLAG_COMPLEMENT, FLAG_SILU, FLAG_RMS_NORM, FLAG_INTERLEAVED, FLAG_ZERO_REST = 128, 256, 512, 1024, 2048
# fault-word bits (KDA_FAULT_* in include/kda.h), read by kda_workspace_faults
FAULT_WAIT_TIMEOUT, FAULT_GATE_RANGE, FAULT_QK_NORM, FAULT_PLACEMENT = 1, 2, 4, 8
# size of the static device scratch behind kda_fwd_noalloc (KDA_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 160 << 20


class KdaError(RuntimeError):
    """A non-zero kda_status_t returned by the library."""

    def __init__(self, status: int, what: str = "kda_fwd"):
        self.status = status
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")


if not os.path.exists(library_path):
    raise ImportError(f"{library_path} is missing; build it with "
                      "`python -c 'import __graft_entry__ as g; g.build()'`")

_lib = ctypes.CDLL(library_path)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_lib.kda_workspace_size.argtypes = [_I64, _I64, _I64]
_lib.kda_workspace_size.restype = ctypes.c_size_t
_lib.kda_is_supported.argtypes = [_I64, _I64, ctypes.c_float]
_lib.kda_is_supported.restype = ctypes.c_int
_lib.kda_status_string.argtypes = [ctypes.c_int]
_lib.kda_status_string.restype = ctypes.c_char_p
_lib.kda_fwd.argtypes = [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P, _P,
                         ctypes.c_float, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_fwd.restype = ctypes.c_int
_lib.kda_fwd_ex.argtypes = [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, ctypes.c_size_t, _P, _P,
                            ctypes.c_float, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.c_uint, _P]
_lib.kda_fwd_ex.restype = ctypes.c_int
_lib.kda_shard_affine.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P, ctypes.c_float,
                                  _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_shard_affine.restype = ctypes.c_int
_lib.kda_shard_scan.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]
_lib.kda_shard_scan.restype = ctypes.c_int
_lib.kda_decode.argtypes = [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, ctypes.c_float, _P, _P,
                            _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_decode.restype = ctypes.c_int
_lib.kda_bwd_workspace_size.argtypes = [_I64, _I64, _I64]
_lib.kda_bwd_workspace_size.restype = ctypes.c_size_t
_lib.kda_bwd.argtypes = [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                         ctypes.c_size_t, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_bwd.restype = ctypes.c_int
_lib.kda_bwd_ex.argtypes = _lib.kda_bwd.argtypes[:-1] + [ctypes.c_uint, _P]
_lib.kda_bwd_ex.restype = ctypes.c_int
_lib.kda_workspace_faults.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), _P]
_lib.kda_workspace_faults.restype = ctypes.c_int
_lib.kda_fwd_noalloc.argtypes = [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, ctypes.c_float, _P, _P, _P,
                                 _I64, _I64, _I64, _I64, _I64, _I64, _P]
_lib.kda_fwd_noalloc.restype = ctypes.c_int
_FN = {}
_I, _U, _F, _SZ = ctypes.c_int, ctypes.c_uint, ctypes.c_float, ctypes.c_size_t
for _name, _args in {
    "kda_glr_fwd": [_P] * 4 + [_SZ, _P, _P, _F, _P, _P, _P, _P] + [_I64] * 5 + [_I, _U, _P],
    "kda_glr_bwd": [_P] * 11 + [_SZ, _P, _P, _F, _P, _P] + [_I64] * 5 + [_I, _U, _P],
    "kda_glr_step": [_P] * 5 + [_F, _P, _P] + [_I64] * 4 + [_I, _U, _P],
    "kda_conv_fwd": [_P, _I64] + [_P] * 6 + [_I64] * 5 + [_I, _U, _P],
    "kda_conv_bwd": [_P, _I64] + [_P] * 9 + [_SZ, _P, _P] + [_I64] * 5 + [_I, _U, _P],
    "kda_conv_step": [_P, _I64] + [_P] * 5 + [_I64] * 4 + [_I, _U, _P],
    "kda_qk_rope_fwd": [_P, _I64, _I64] * 2 + [_P] * 6 + [_F] + [_I64] * 5 + [_I, _U, _P],
    "kda_qk_rope_bwd": [_P, _I64, _I64] * 2 + [_P] * 7 + [_SZ] + [_P] * 4 + [_F] + [_I64] * 5 + [_I, _U, _P],
    "kda_la_fwd": [_P, _I64, _I64] * 3 + [_P, _F, _P, _P, _SZ, _P, _P, _P] + [_I64] * 6 + [_U, _P],
    "kda_la_bwd": [_P, _I64, _I64] * 3 + [_P, _F] + [_P] * 8 + [_SZ, _P, _P] + [_I64] * 6 + [_U, _P],
    "kda_la_step": [_P, _I64, _I64] * 3 + [_P, _F, _P, _P, _P] + [_I64] * 5 + [_P],
    "kda_attn_fwd": [_P, _I64, _I64] * 3 + [_F, _P, _P, _P, _P, _SZ, _P, _P] + [_I64] * 7 + [_U, _P],
    "kda_attn_bwd": [_P, _I64, _I64] * 3 + [_F] + [_P] * 9 + [_SZ, _P, _P] + [_I64] * 7 + [_U, _P],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _I
    _FN[_name] = getattr(_lib, _name)
for _name, _n in {"kda_glr_workspace_size": 3, "kda_glr_states_size": 3, "kda_glr_bwd_workspace_size": 3,
                  "kda_conv_bwd_workspace_size": 3, "kda_qk_rope_bwd_workspace_size": 4,
                  "kda_la_workspace_size": 4, "kda_la_bwd_workspace_size": 5,
                  "kda_attn_workspace_size": 6, "kda_attn_bwd_workspace_size": 6}.items():
    getattr(_lib, _name).argtypes = [_I64] * _n
    getattr(_lib, _name).restype = _SZ


def kda_workspace_size(T: int, H: int, N: int) -> int:
    """Workspace bytes for T packed tokens, H heads and N sequences."""
    return int(_lib.kda_workspace_size(T, H, N))


def kda_is_supported(K: int, V: int, lower_bound: float) -> bool:
    return bool(_lib.kda_is_supported(K, V, lower_bound))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_inputs(q, k, v, raw_gate, raw_beta, out, A_log, dt_bias, cu_seqlens):
    B, T, H, K = q.shape
    V = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("raw_gate", raw_gate), ("raw_beta", raw_beta),
                    ("out", out)):
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda):
            raise ValueError(f"{name} must be a contiguous bf16 device tensor")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda):
            raise ValueError(f"{name} must be a contiguous fp32 device tensor")
    if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda):
        raise ValueError("cu_seqlens must be an int32 device tensor")
    if tuple(k.shape) != (B, T, H, K) or tuple(raw_gate.shape) != (B, T, H, K) or \
            tuple(v.shape) != (B, T, H, V) or (out is not None and tuple(out.shape) != (B, T, H, V)) or \
            tuple(raw_beta.shape) != (B, T, H):
        raise ValueError("inconsistent q/k/v/raw_gate/raw_beta/out shapes")
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    return B, T, H, K, V, N


def _check_f32(name, t, shape):
    if t is None:
        return
    if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous fp32 device tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")


def _stream(stream, dev):
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    return ctypes.c_void_p(int(stream))


def kda_fwd(q, k, v, raw_gate, raw_beta, scale, out, workspace, A_log, dt_bias, lower_bound,
            initial_state=None, final_state=None, cu_seqlens=None, stream=None):
    """Enqueue one KDA forward on ``stream`` (default: torch's current stream).

    Tensors are torch device tensors in the layouts of include/kda.h:
    q, k, raw_gate bf16 [B,T,H,K]; v and out bf16 [B,T,H,V]; raw_beta bf16 [B,T,H];
    workspace uint8 [>= kda_workspace_size(B*T, H, N)]; A_log fp32 [H];
    dt_bias fp32 [H,K]; initial_state / final_state fp32 [N,H,K,V] or None;
    cu_seqlens int32 [N+1] or None.  Raises KdaError on a non-zero status.
    """
    if out is None:
        raise ValueError("out is required")
    B, T, H, K, V, N = _check_inputs(q, k, v, raw_gate, raw_beta, out, A_log, dt_bias, cu_seqlens)
    _check_f32("initial_state", initial_state, (N, H, K, V))
    _check_f32("final_state", final_state, (N, H, K, V))
    rc = _lib.kda_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), float(scale),
                      _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                      _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(initial_state),
                      _ptr(final_state), _ptr(cu_seqlens), B, T, H, K, V, N, _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc)


def kda_fwd_noalloc(q, k, v, raw_gate, raw_beta, scale, out, A_log, dt_bias, lower_bound,
                    initial_state=None, final_state=None, cu_seqlens=None, stream=None):
    """kda_fwd without a workspace: the library's static per-GPU scratch of
    NOALLOC_SCRATCH_BYTES is used instead (calls larger than it raise KdaError with
    KDA_ERR_WORKSPACE; calls that overlap on one GPU race)."""
    if out is None:
        raise ValueError("out is required")
    B, T, H, K, V, N = _check_inputs(q, k, v, raw_gate, raw_beta, out, A_log, dt_bias, cu_seqlens)
    _check_f32("initial_state", initial_state, (N, H, K, V))
    _check_f32("final_state", final_state, (N, H, K, V))
    rc = _lib.kda_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), float(scale),
                              _ptr(out), _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(initial_state),
                              _ptr(final_state), _ptr(cu_seqlens), B, T, H, K, V, N, _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc, "kda_fwd_noalloc")


def kda_fwd_ex(q, k, v, raw_gate, raw_beta, scale, out, workspace, A_log, dt_bias, lower_bound,
               initial_state=None, final_state=None, cu_seqlens=None, flags=0, stream=None):
    """kda_fwd with variant flags (an OR of the FLAG_* bits).  With FLAG_GATE_GIVEN,
    A_log and dt_bias may be None; with FLAG_STATE_VK the states are [N,H,V,K];
    FLAG_KEEP_RECORDS leaves every chunk record in the workspace, and
    FLAG_REUSE_RECORDS skips the intra-chunk pass and uses the records that such a
    previous call on this workspace (same inputs but v and the states) left there."""
    if out is None:
        raise ValueError("out is required")
    if not flags & FLAG_GATE_GIVEN and (A_log is None or dt_bias is None):
        raise ValueError("A_log and dt_bias are required unless FLAG_GATE_GIVEN")
    B, T, H, K, V, N = _check_inputs(q, k, v, raw_gate, raw_beta, out, A_log, dt_bias, cu_seqlens)
    st_shape = (N, H, V, K) if flags & FLAG_STATE_VK else (N, H, K, V)
    _check_f32("initial_state", initial_state, st_shape)
    _check_f32("final_state", final_state, st_shape)
    rc = _lib.kda_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), float(scale),
                         _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                         _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(initial_state),
                         _ptr(final_state), _ptr(cu_seqlens), B, T, H, K, V, N, int(flags),
                         _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc, "kda_fwd_ex")


def kda_shard_affine(q, k, v, raw_gate, raw_beta, workspace, A_log, dt_bias, lower_bound, P, R,
                     cu_seqlens=None, stream=None):
    """Enqueue the per-shard affine maps: every sequence n of the call (a shard)
    takes an entering state S to P[n] S + R[n].  P fp32 [N,H,K,K], R fp32 [N,H,K,V]."""
    B, T, H, K, V, N = _check_inputs(q, k, v, raw_gate, raw_beta, None, A_log, dt_bias, cu_seqlens)
    _check_f32("P", P, (N, H, K, K))
    _check_f32("R", R, (N, H, K, V))
    rc = _lib.kda_shard_affine(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(A_log), _ptr(dt_bias),
                               float(lower_bound), _ptr(P), _ptr(R), _ptr(cu_seqlens), B, T, H, K, V, N,
                               _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc, "kda_shard_affine")


def kda_shard_scan(P, R, starts, initial_state=None, final_state=None, stream=None):
    """Enqueue the fold over consecutive shards: starts[0] = initial_state (or 0),
    starts[r+1] = P[r] starts[r] + R[r]; final_state gets the state after the last shard."""
    n, H, K, _ = P.shape
    V = R.shape[-1]
    _check_f32("P", P, (n, H, K, K))
    _check_f32("R", R, (n, H, K, V))
    _check_f32("starts", starts, (n, H, K, V))
    _check_f32("initial_state", initial_state, (H, K, V))
    _check_f32("final_state", final_state, (H, K, V))
    rc = _lib.kda_shard_scan(_ptr(P), _ptr(R), _ptr(initial_state), _ptr(starts), _ptr(final_state),
                             n, H, K, V, _stream(stream, P.device))
    if rc != 0:
        raise KdaError(rc, "kda_shard_scan")


def kda_decode(q, k, v, raw_gate, raw_beta, scale, out, A_log, dt_bias, lower_bound,
               initial_state=None, final_state=None, stream=None):
    """Enqueue the token-by-token step over B sequences of T tokens (layouts as for
    kda_fwd, states fp32 [B,H,K,V]; final_state may be initial_state for an in-place
    update).  Raises KdaError on a non-zero status."""
    if out is None:
        raise ValueError("out is required")
    B, T, H, K, V, _ = _check_inputs(q, k, v, raw_gate, raw_beta, out, A_log, dt_bias, None)
    _check_f32("initial_state", initial_state, (B, H, K, V))
    _check_f32("final_state", final_state, (B, H, K, V))
    rc = _lib.kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), float(scale), _ptr(out),
                         _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(initial_state),
                         _ptr(final_state), B, T, H, K, V, _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc, "kda_decode")


def kda_bwd_workspace_size(T: int, H: int, N: int) -> int:
    """Workspace bytes of kda_bwd for T packed tokens, H heads and N sequences."""
    return int(_lib.kda_bwd_workspace_size(T, H, N))


def kda_bwd(q, k, v, raw_gate, raw_beta, scale, d_out, dq, dk, dv, d_raw_gate, d_raw_beta, dA_log,
            d_dt_bias, workspace, A_log, dt_bias, lower_bound, initial_state=None, d_final=None,
            d_initial_state=None, cu_seqlens=None, stream=None):
    """Enqueue the gradients of one KDA forward (same inputs as kda_fwd) for the output
    gradient d_out (bf16 [B,T,H,V]) and the final-state gradient d_final (fp32 [N,H,K,V]
    or None for zero).  Writes dq, dk, d_raw_gate (bf16 [B,T,H,K]), dv (bf16 [B,T,H,V]),
    d_raw_beta (bf16 [B,T,H]), dA_log (fp32 [H]), d_dt_bias (fp32 [H,K]) and, if given,
    d_initial_state (fp32 [N,H,K,V])."""
    kda_bwd_ex(q, k, v, raw_gate, raw_beta, scale, d_out, dq, dk, dv, d_raw_gate, d_raw_beta, dA_log,
               d_dt_bias, workspace, A_log, dt_bias, lower_bound, initial_state, d_final, d_initial_state,
               cu_seqlens, flags=0, stream=stream, _name="kda_bwd")


def kda_bwd_ex(q, k, v, raw_gate, raw_beta, scale, d_out, dq, dk, dv, d_raw_gate, d_raw_beta, dA_log,
               d_dt_bias, workspace, A_log, dt_bias, lower_bound, initial_state=None, d_final=None,
               d_initial_state=None, cu_seqlens=None, flags=0, stream=None, _name="kda_bwd_ex"):
    """kda_bwd for the variants of kda_fwd_ex (an OR of the FLAG_* bits).  With
    FLAG_GATE_GIVEN, A_log, dt_bias, dA_log and d_dt_bias may be None; with FLAG_STATE_VK
    the states and their gradients are [N,H,V,K]."""
    if not flags & FLAG_GATE_GIVEN and (A_log is None or dt_bias is None or dA_log is None or d_dt_bias is None):
        raise ValueError("A_log, dt_bias, dA_log and d_dt_bias are required unless FLAG_GATE_GIVEN")
    B, T, H, K, V, N = _check_inputs(q, k, v, raw_gate, raw_beta, d_out, A_log, dt_bias, cu_seqlens)
    _check_inputs(q, dk, dv, d_raw_gate, d_raw_beta, None, None, None, None)
    if tuple(dq.shape) != tuple(q.shape) or dq.dtype != torch.bfloat16 or not dq.is_contiguous():
        raise ValueError("dq must be a contiguous bf16 tensor shaped like q")
    st_shape = (N, H, V, K) if flags & FLAG_STATE_VK else (N, H, K, V)
    _check_f32("initial_state", initial_state, st_shape)
    _check_f32("d_final", d_final, st_shape)
    _check_f32("d_initial_state", d_initial_state, st_shape)
    _check_f32("dA_log", dA_log, (H,))
    _check_f32("d_dt_bias", d_dt_bias, (H, K))
    rc = _lib.kda_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(raw_gate), _ptr(raw_beta), float(scale), _ptr(d_out),
                         _ptr(d_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(d_raw_gate), _ptr(d_raw_beta),
                         _ptr(dA_log), _ptr(d_dt_bias), _ptr(d_initial_state), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _ptr(A_log), _ptr(dt_bias),
                         float(lower_bound), _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N,
                         int(flags), _stream(stream, q.device))
    if rc != 0:
        raise KdaError(rc, _name)


def kda_workspace_faults(workspace, stream=None) -> int:
    """The fault word (an OR of the FAULT_* bits) of the last call on ``workspace``,
    read after the work enqueued on ``stream`` has finished (this synchronises it)."""
    word = ctypes.c_uint32(0)
    rc = _lib.kda_workspace_faults(_ptr(workspace), ctypes.byref(word), _stream(stream, workspace.device))
    if rc != 0:
        raise KdaError(rc, "kda_workspace_faults")
    return int(word.value)


# ---------------------------------------------------------------------------
# operators around the core
# ---------------------------------------------------------------------------
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}


class _Call:
    """The checks and the stream of one call: tensors on one GPU, of a type, contiguous, of a shape."""

    __slots__ = ("index",)

    def __init__(self, first, name):
        self.index = first.get_device()
        if self.index < 0:
            raise ValueError(f"{name} must be a device tensor")

    def token(self, t, name, dtype, shape=None, contiguous=True):
        if t.dtype is not dtype or t.get_device() != self.index or (contiguous and not t.is_contiguous()):
            raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}{dtype} tensor on cuda:{self.index}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}")
        return t.data_ptr()

    def option(self, t, name, dtype, shape=None):
        return None if t is None else self.token(t, name, dtype, shape)

    def run(self, what, stream, *args):
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self.index)
        fn = _FN[what]
        if torch._C._cuda_getDevice() == self.index:
            rc = fn(*args, stream)
        else:  # a launch goes to the current device
            with torch.cuda.device(self.index):
                rc = fn(*args, stream)
        if rc != 0:
            raise KdaError(rc, what)


def _type_of(t, name):
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be bf16 or fp32")
    return _DTYPE[t.dtype]


def _sequences(cu_seqlens, c, B):
    if cu_seqlens is None:
        return B, None
    return cu_seqlens.numel() - 1, c.token(cu_seqlens, "cu_seqlens", torch.int32)


def _bytes(c, workspace):
    if workspace.get_device() != c.index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{c.index}")
    return workspace.data_ptr(), workspace.nbytes


def kda_glr_workspace_size(T: int, H: int, K: int) -> int:
    """Workspace bytes of kda_glr_fwd for T packed tokens, H heads of K channels."""
    return int(_lib.kda_glr_workspace_size(T, H, K))


def kda_glr_states_size(T: int, H: int, K: int) -> int:
    """Bytes of the states that kda_glr_fwd leaves for kda_glr_bwd."""
    return int(_lib.kda_glr_states_size(T, H, K))


def kda_glr_bwd_workspace_size(T: int, H: int, K: int) -> int:
    """Workspace bytes of kda_glr_bwd for T packed tokens, H heads of K channels."""
    return int(_lib.kda_glr_bwd_workspace_size(T, H, K))


def _states(c, states, need):
    if states is None:
        return None
    if states.numel() * states.element_size() < need:
        raise ValueError(f"states must hold {need} bytes")
    return c.token(states, "states", states.dtype)


def _glr(x, raw_gate, A_log, dt_bias, flags, name):
    c = _Call(x, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, K]")
    B, T, H, K = x.shape
    ty = _type_of(x, "x")
    if not flags & FLAG_GATE_GIVEN and (A_log is None or dt_bias is None):
        raise ValueError("A_log and dt_bias are required unless FLAG_GATE_GIVEN")
    return (c, ty, B, T, H, K, c.token(x, "x", x.dtype), c.token(raw_gate, "raw_gate", x.dtype, x.shape),
            c.option(A_log, "A_log", torch.float32, (H,)), c.option(dt_bias, "dt_bias", torch.float32, (H, K)))


def kda_glr_fwd(x, raw_gate, out, workspace, A_log, dt_bias, lower_bound, initial_state=None, final_state=None,
                states=None, cu_seqlens=None, flags=0, stream=None):
    """Enqueue the gated linear recurrence h_t = a_t h_{t-1} + b_t x_t on ``stream`` (default:
    torch's current stream), a_t = exp(g_t) under KDA's gate, b_t = 1 or 1 - a_t.

    x, raw_gate, out bf16 or fp32 [B,T,H,K]; workspace >= kda_glr_workspace_size(B*T, H, K) bytes;
    A_log fp32 [H], dt_bias fp32 [H,K] (None with FLAG_GATE_GIVEN); initial_state / final_state
    fp32 [N,H,K] or None; states >= kda_glr_states_size(B*T, H, K) bytes if kda_glr_bwd follows;
    cu_seqlens int32 [N+1] or None; flags an OR of FLAG_GATE_GIVEN, FLAG_COMPLEMENT
    and FLAG_ZERO_REST."""
    c, ty, B, T, H, K, px, pg, pa, pd = _glr(x, raw_gate, A_log, dt_bias, flags, "kda_glr_fwd")
    N, pcu = _sequences(cu_seqlens, c, B)
    ws, size = _bytes(c, workspace)
    c.run("kda_glr_fwd", stream, px, pg, c.token(out, "out", x.dtype, x.shape), ws, size, pa, pd, float(lower_bound),
          c.option(initial_state, "initial_state", torch.float32, (N, H, K)),
          c.option(final_state, "final_state", torch.float32, (N, H, K)),
          _states(c, states, kda_glr_states_size(B * T, H, K)), pcu, B, T, H, K, N, ty, int(flags))


def kda_glr_bwd(x, raw_gate, states, d_out, dx, d_raw_gate, dA_log, d_dt_bias, workspace, A_log, dt_bias,
                lower_bound, initial_state=None, d_final=None, d_initial_state=None, cu_seqlens=None, flags=0,
                stream=None):
    """Enqueue the gradients of a kda_glr_fwd call with the same inputs, which left ``states``, for
    d_out [B,T,H,K] and d_final (fp32 [N,H,K] or None for zero).  Writes dx, d_raw_gate, dA_log
    and d_dt_bias (None with FLAG_GATE_GIVEN) and, if given, d_initial_state; workspace >=
    kda_glr_bwd_workspace_size(B*T, H, K) bytes."""
    c, ty, B, T, H, K, px, pg, pa, pd = _glr(x, raw_gate, A_log, dt_bias, flags, "kda_glr_bwd")
    N, pcu = _sequences(cu_seqlens, c, B)
    ws, size = _bytes(c, workspace)
    c.run("kda_glr_bwd", stream, px, pg, _states(c, states, kda_glr_states_size(B * T, H, K)),
          c.token(d_out, "d_out", x.dtype, x.shape), c.option(d_final, "d_final", torch.float32, (N, H, K)),
          c.token(dx, "dx", x.dtype, x.shape), c.token(d_raw_gate, "d_raw_gate", x.dtype, x.shape),
          c.option(dA_log, "dA_log", torch.float32, (H,)), c.option(d_dt_bias, "d_dt_bias", torch.float32, (H, K)),
          c.option(d_initial_state, "d_initial_state", torch.float32, (N, H, K)), ws, size, pa, pd,
          float(lower_bound), c.option(initial_state, "initial_state", torch.float32, (N, H, K)), pcu, B, T, H, K, N,
          ty, int(flags))


def kda_glr_step(x, raw_gate, out, A_log, dt_bias, lower_bound, initial_state=None, final_state=None, flags=0,
                 stream=None):
    """Enqueue the recurrence over B sequences of T tokens each (decoding): one launch, no workspace;
    states fp32 [B,H,K], final_state may be initial_state for an in-place update."""
    c, ty, B, T, H, K, px, pg, pa, pd = _glr(x, raw_gate, A_log, dt_bias, flags, "kda_glr_step")
    c.run("kda_glr_step", stream, px, pg, c.token(out, "out", x.dtype, x.shape), pa, pd, float(lower_bound),
          c.option(initial_state, "initial_state", torch.float32, (B, H, K)),
          c.option(final_state, "final_state", torch.float32, (B, H, K)), B, T, H, K, ty, int(flags))


def _row_stride(t, name):
    """Elements between tokens of a [B, T, ...] tensor whose rows lie evenly: a slice of a wider one."""
    B, T = t.shape[:2]
    st = t.stride()
    if T > 1:
        if B > 1 and st[0] != T * st[1]:
            raise ValueError(f"{name}: the tokens of all sequences must lie evenly apart")
        return st[1]
    return st[0] if B > 1 else math.prod(t.shape[2:])


def _conv(x, weight, bias, flags):
    c = _Call(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    if C > 1 and x.stride(2) != 1:
        raise ValueError("the channels of x must be contiguous")
    return (c, _type_of(x, "x"), B, T, C, W, c.token(x, "x", x.dtype, contiguous=False), _row_stride(x, "x"),
            c.token(weight, "weight", torch.float32, (C, W)), c.option(bias, "bias", torch.float32, (C,)))


def kda_conv_fwd(x, weight, out, bias=None, initial_state=None, final_state=None, cu_seqlens=None, flags=0,
                 stream=None):
    """Enqueue the short causal depthwise convolution z_t = bias + sum_j weight[:, j] x_{t-(W-1)+j},
    followed by z sigmoid(z) with FLAG_SILU.

    x bf16 or fp32 [B,T,C], its tokens evenly apart (a slice of a wider tensor will do); weight
    fp32 [C,W], W 2 to 4; bias fp32 [C] or None; out [B,T,C]; initial_state / final_state
    [N,W-1,C] of x's type, the last W-1 inputs, or None; cu_seqlens int32 [N+1] or None."""
    c, ty, B, T, C, W, px, xs, pw, pb = _conv(x, weight, bias, flags)
    N, pcu = _sequences(cu_seqlens, c, B)
    c.run("kda_conv_fwd", stream, px, xs, pw, pb, c.token(out, "out", x.dtype, x.shape),
          c.option(initial_state, "initial_state", x.dtype, (N, W - 1, C)),
          c.option(final_state, "final_state", x.dtype, (N, W - 1, C)), pcu, B, T, C, W, N, ty, int(flags))


def kda_conv_bwd_workspace_size(T: int, C: int, W: int) -> int:
    """Workspace bytes of kda_conv_bwd for T packed tokens of C channels and W taps."""
    return int(_lib.kda_conv_bwd_workspace_size(T, C, W))


def kda_conv_bwd(x, weight, d_out, dx, d_weight, workspace, bias=None, d_bias=None, initial_state=None, d_final=None,
                 d_initial_state=None, cu_seqlens=None, flags=0, stream=None):
    """Enqueue the gradients of a kda_conv_fwd call with the same inputs: dx [B,T,C], d_weight fp32
    [C,W], d_bias fp32 [C] and d_initial_state [N,W-1,C] (None to skip), for d_out [B,T,C] and
    d_final [N,W-1,C] (None for zero); workspace >= kda_conv_bwd_workspace_size(B*T, C, W) bytes."""
    c, ty, B, T, C, W, px, xs, pw, pb = _conv(x, weight, bias, flags)
    N, pcu = _sequences(cu_seqlens, c, B)
    ws, size = _bytes(c, workspace)
    st = (N, W - 1, C)
    c.run("kda_conv_bwd", stream, px, xs, pw, pb, c.token(d_out, "d_out", x.dtype, x.shape),
          c.option(d_final, "d_final", x.dtype, st), c.token(dx, "dx", x.dtype, x.shape),
          c.token(d_weight, "d_weight", torch.float32, (C, W)), c.option(d_bias, "d_bias", torch.float32, (C,)),
          c.option(d_initial_state, "d_initial_state", x.dtype, st), ws, size,
          c.option(initial_state, "initial_state", x.dtype, st), pcu, B, T, C, W, N, ty, int(flags))


def kda_conv_step(x, weight, out, bias=None, initial_state=None, final_state=None, flags=0, stream=None):
    """Enqueue the convolution over B sequences of T tokens each (decoding); states [B,W-1,C] of x's
    type, final_state may be initial_state for an in-place update."""
    c, ty, B, T, C, W, px, xs, pw, pb = _conv(x, weight, bias, flags)
    c.run("kda_conv_step", stream, px, xs, pw, pb, c.token(out, "out", x.dtype, x.shape),
          c.option(initial_state, "initial_state", x.dtype, (B, W - 1, C)),
          c.option(final_state, "final_state", x.dtype, (B, W - 1, C)), B, T, C, W, ty, int(flags))


def _qk(q, k, positions, inv_freq, q_weight, k_weight):
    c = _Call(q, "q")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, H, D]")
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    ptrs = []
    for t, name, H in ((q, "q", Hq), (k, "k", Hk)):
        p = c.token(t, name, q.dtype, (B, T, H, D), contiguous=False)
        if D > 1 and t.stride(3) != 1:
            raise ValueError(f"the channels of {name} must be contiguous")
        ptrs += [p, _row_stride(t, name), t.stride(2) if H > 1 else D]
    R = 0
    if inv_freq is not None and inv_freq.numel():
        R = 2 * inv_freq.numel()
        if positions is None:
            raise ValueError("positions are required with inv_freq")
    return (c, _type_of(q, "q"), B, T, Hq, Hk, D, R, ptrs,
            c.option(q_weight, "q_weight", torch.float32, (D,)), c.option(k_weight, "k_weight", torch.float32, (D,)),
            c.option(positions, "positions", torch.int32, (B, T)),
            c.option(inv_freq, "inv_freq", torch.float64, (R // 2,)))


def kda_qk_rope_fwd(q, k, q_out, k_out, positions, inv_freq, eps=1e-6, q_weight=None, k_weight=None, flags=0,
                    stream=None):
    """Enqueue the norm of q and k per head (L2, as in the core; FLAG_RMS_NORM; none with
    FLAG_NO_QK_NORM), the product with q_weight / k_weight (fp32 [D] or None) and the rotation of
    the first R = 2 * inv_freq.numel() channels by positions * inv_freq.

    q [B,T,Hq,D], k [B,T,Hk,D] bf16 or fp32, tokens and heads evenly apart; q_out, k_out contiguous,
    or q and k themselves for an in-place call; positions int32 [B,T]; inv_freq fp64 [R/2]
    (None: no rotation).  FLAG_INTERLEAVED rotates the pairs (2i, 2i+1)."""
    c, ty, B, T, Hq, Hk, D, R, p, pqw, pkw, ppos, pf = _qk(q, k, positions, inv_freq, q_weight, k_weight)
    po = [c.token(o, n, q.dtype, t.shape, contiguous=o.data_ptr() != t.data_ptr())
          for o, n, t in ((q_out, "q_out", q), (k_out, "k_out", k))]
    if any(o.data_ptr() == t.data_ptr() and o.numel() and o.stride() != t.stride() for o, t in ((q_out, q), (k_out, k))):
        raise ValueError("an in-place output must be the input itself")
    c.run("kda_qk_rope_fwd", stream, *p, *po, pqw, pkw, ppos, pf, float(eps), B * T, Hq, Hk, D, R, ty, int(flags))


def kda_qk_rope_bwd_workspace_size(tokens: int, Hq: int, Hk: int, D: int) -> int:
    """Workspace bytes of kda_qk_rope_bwd where weight gradients are asked for."""
    return int(_lib.kda_qk_rope_bwd_workspace_size(tokens, Hq, Hk, D))


def kda_qk_rope_bwd(q, k, d_q_out, d_k_out, dq, dk, positions, inv_freq, eps=1e-6, q_weight=None, k_weight=None,
                    d_q_weight=None, d_k_weight=None, workspace=None, flags=0, stream=None):
    """Enqueue the gradients of a kda_qk_rope_fwd call with the same inputs: dq, dk (contiguous, may
    be d_q_out and d_k_out) and, if given, d_q_weight and d_k_weight (fp32 [D]), which need a
    workspace of kda_qk_rope_bwd_workspace_size(B*T, Hq, Hk, D) bytes."""
    c, ty, B, T, Hq, Hk, D, R, p, pqw, pkw, ppos, pf = _qk(q, k, positions, inv_freq, q_weight, k_weight)
    ws, size = (None, 0) if workspace is None else _bytes(c, workspace)
    c.run("kda_qk_rope_bwd", stream, *p, c.token(d_q_out, "d_q_out", q.dtype, q.shape),
          c.token(d_k_out, "d_k_out", q.dtype, k.shape), c.token(dq, "dq", q.dtype, q.shape),
          c.token(dk, "dk", q.dtype, k.shape), c.option(d_q_weight, "d_q_weight", torch.float32, (D,)),
          c.option(d_k_weight, "d_k_weight", torch.float32, (D,)), ws, size, pqw, pkw, ppos, pf, float(eps), B * T,
          Hq, Hk, D, R, ty, int(flags))


# ---------------------------------------------------------------------------
# token mixers beside the core
# ---------------------------------------------------------------------------
def _heads(c, t, name, shape):
    """Pointer, token stride and head stride of a bf16 token array [B, T, H, channels] whose tokens and
    heads lie evenly apart."""
    p = c.token(t, name, torch.bfloat16, shape, contiguous=False)
    if t.is_contiguous():
        return p, shape[2] * shape[3], shape[3]
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return p, _row_stride(t, name), t.stride(2) if t.shape[2] > 1 else t.shape[3]


def _la(q, k, v, log_decay):
    c = _Call(q, "q")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, T, H, channels]")
    B, T, H, K = q.shape
    V = v.shape[3]
    return c, B, T, H, K, V, [*_heads(c, q, "q", q.shape), *_heads(c, k, "k", q.shape),
                              *_heads(c, v, "v", (B, T, H, V)), c.token(log_decay, "log_decay", torch.float32, (H,))]


def kda_la_workspace_size(T: int, H: int, K: int, V: int) -> int:
    """Workspace bytes of kda_la_fwd for T packed tokens and H heads of K and V channels (0: none needed)."""
    return int(_lib.kda_la_workspace_size(T, H, K, V))


def kda_la_bwd_workspace_size(T: int, H: int, K: int, V: int, N: int) -> int:
    """Workspace bytes of kda_la_bwd for T packed tokens, H heads of K and V channels and N sequences."""
    return int(_lib.kda_la_bwd_workspace_size(T, H, K, V, N))


def kda_la_fwd(q, k, v, log_decay, scale, out, workspace, initial_state=None, final_state=None, cu_seqlens=None, flags=0,
               stream=None):
    """Enqueue linear attention with a decay for each head, S_t = exp(log_decay) S_{t-1} + k_t v_t^T,
    out_t = scale S_t^T q_t, on ``stream`` (default: torch's current stream).

    q, k bf16 [B,T,H,K], v bf16 [B,T,H,V], tokens and heads evenly apart; K and V 64 or 128; log_decay
    fp32 [H], at most 0; out bf16 [B,T,H,V]; workspace >= kda_la_workspace_size(B*T, H, K, V) bytes (None if that is 0);
    initial_state / final_state fp32 [N,H,K,V] or None; cu_seqlens int32 [N+1] or None; flags 0 or
    FLAG_ZERO_REST."""
    c, B, T, H, K, V, p = _la(q, k, v, log_decay)
    N, pcu = _sequences(cu_seqlens, c, B)
    ws, size = (None, 0) if workspace is None else _bytes(c, workspace)
    st = (N, H, K, V)
    c.run("kda_la_fwd", stream, *p, float(scale), c.token(out, "out", torch.bfloat16, v.shape), ws, size,
          c.option(initial_state, "initial_state", torch.float32, st),
          c.option(final_state, "final_state", torch.float32, st), pcu, B, T, H, K, V, N, int(flags))


def kda_la_bwd(q, k, v, log_decay, scale, d_out, dq, dk, dv, workspace, d_log_decay=None, initial_state=None, d_final=None,
               d_initial_state=None, cu_seqlens=None, flags=0, stream=None):
    """Enqueue the gradients of a kda_la_fwd call with the same inputs, for d_out bf16 [B,T,H,V] and
    d_final (fp32 [N,H,K,V], None for zero).  Writes dq, dk, dv (bf16, contiguous) and, if given,
    d_log_decay (fp32 [H]) and d_initial_state; workspace >= kda_la_bwd_workspace_size(B*T, H, K, V, N)
    bytes."""
    c, B, T, H, K, V, p = _la(q, k, v, log_decay)
    N, pcu = _sequences(cu_seqlens, c, B)
    ws, size = _bytes(c, workspace)
    st, bf = (N, H, K, V), torch.bfloat16
    c.run("kda_la_bwd", stream, *p, float(scale), c.token(d_out, "d_out", bf, v.shape),
          c.option(d_final, "d_final", torch.float32, st), c.token(dq, "dq", bf, q.shape), c.token(dk, "dk", bf, q.shape),
          c.token(dv, "dv", bf, v.shape), c.option(d_log_decay, "d_log_decay", torch.float32, (H,)),
          c.option(d_initial_state, "d_initial_state", torch.float32, st), ws, size,
          c.option(initial_state, "initial_state", torch.float32, st), pcu, B, T, H, K, V, N, int(flags))


def kda_la_step(q, k, v, log_decay, scale, out, initial_state=None, final_state=None, stream=None):
    """Enqueue linear attention over B sequences of T tokens each (decoding): one launch, no workspace;
    states fp32 [B,H,K,V], final_state may be initial_state for an in-place update."""
    c, B, T, H, K, V, p = _la(q, k, v, log_decay)
    st = (B, H, K, V)
    c.run("kda_la_step", stream, *p, float(scale), c.token(out, "out", torch.bfloat16, v.shape),
          c.option(initial_state, "initial_state", torch.float32, st),
          c.option(final_state, "final_state", torch.float32, st), B, T, H, K, V)


def _attn(q, k, v, cu_seqlens_q, cu_seqlens_k):
    c = _Call(q, "q")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [B, T, H, D]")
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    p = [*_heads(c, q, "q", q.shape), *_heads(c, k, "k", (B, Tk, Hk, D)), *_heads(c, v, "v", (B, Tk, Hk, D))]
    if (cu_seqlens_q is None) != (cu_seqlens_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k go together")
    N, pq = _sequences(cu_seqlens_q, c, B)
    Nk, pk = _sequences(cu_seqlens_k, c, B)
    if N != Nk:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    return c, (B, Tq, Tk, Hq, Hk, D, N), p, pq, pk


def kda_attn_workspace_size(Tq: int, Tk: int, Hq: int, Hk: int, D: int, N: int) -> int:
    """Workspace bytes of kda_attn_fwd for Tq packed queries and Tk packed keys of N sequences (0: none needed)."""
    return int(_lib.kda_attn_workspace_size(Tq, Tk, Hq, Hk, D, N))


def kda_attn_bwd_workspace_size(Tq: int, Tk: int, Hq: int, Hk: int, D: int, N: int) -> int:
    """Workspace bytes of kda_attn_bwd for Tq packed queries and Tk packed keys of N sequences."""
    return int(_lib.kda_attn_bwd_workspace_size(Tq, Tk, Hq, Hk, D, N))


def kda_attn_fwd(q, k, v, scale, out, lse, workspace, out_lo=None, cu_seqlens_q=None, cu_seqlens_k=None, flags=0,
                 stream=None):
    """Enqueue causal softmax attention on ``stream`` (default: torch's current stream): query i of a
    sequence of nq queries and nk keys sees the keys j <= i + nk - nq.

    q bf16 [B,Tq,Hq,D], k, v bf16 [B,Tk,Hk,D], tokens and heads evenly apart (the first Tk rows of a longer
    cache only with B = 1), D 64 or 128, Hq a multiple of Hk; out bf16 [B,Tq,Hq,D]; out_lo the same for kda_attn_bwd (what out's rounding took off), or
    None; lse fp32 [B,Tq,Hq]; workspace >= kda_attn_workspace_size(B*Tq, B*Tk, Hq,
    Hk, D, N) bytes (None if that is 0); cu_seqlens_q, cu_seqlens_k int32 [N+1] (the same one for prompts without a past)
    or None; flags 0 or FLAG_ZERO_REST."""
    c, sizes, p, pq, pk = _attn(q, k, v, cu_seqlens_q, cu_seqlens_k)
    ws, size = (None, 0) if workspace is None else _bytes(c, workspace)
    c.run("kda_attn_fwd", stream, *p, float(scale), c.token(out, "out", torch.bfloat16, q.shape),
          c.option(out_lo, "out_lo", torch.bfloat16, q.shape), c.token(lse, "lse", torch.float32, q.shape[:3]), ws, size, pq, pk, *sizes, int(flags))


def kda_attn_bwd(q, k, v, scale, out, out_lo, lse, d_out, dq, dk, dv, workspace, d_lse=None, cu_seqlens_q=None,
                 cu_seqlens_k=None, flags=0, stream=None):
    """Enqueue the gradients of a kda_attn_fwd call with the same inputs, which wrote out, out_lo and lse,
    for d_out bf16 [B,Tq,Hq,D] and d_lse (fp32 [B,Tq,Hq], None for zero).  Writes dq, dk and dv (bf16,
    contiguous); workspace >= kda_attn_bwd_workspace_size(B*Tq, B*Tk, Hq, Hk, D, N) bytes."""
    c, sizes, p, pq, pk = _attn(q, k, v, cu_seqlens_q, cu_seqlens_k)
    ws, size = _bytes(c, workspace)
    bf, ls = torch.bfloat16, q.shape[:3]
    c.run("kda_attn_bwd", stream, *p, float(scale), c.token(out, "out", bf, q.shape),
          c.token(out_lo, "out_lo", bf, q.shape), c.token(lse, "lse", torch.float32, ls), c.token(d_out, "d_out", bf, q.shape),
          c.option(d_lse, "d_lse", torch.float32, ls), c.token(dq, "dq", bf, q.shape), c.token(dk, "dk", bf, k.shape),
          c.token(dv, "dv", bf, k.shape), ws, size, pq, pk, *sizes, int(flags))


def raw_call(*args):
    """Call the C entry point with already-marshalled ctypes arguments (tests)."""
    return _lib.kda_fwd(*args)
