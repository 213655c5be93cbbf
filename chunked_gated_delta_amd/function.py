"""Differentiable KDA operators for PyTorch training code.

``kda_chunk`` is the chunked forward; ``kda_glr`` the gated linear recurrence,
``kda_short_conv`` the short causal convolution and ``kda_qk_norm_rope`` the
norm and rotation of queries and keys.  Each allocates its outputs and
workspaces with PyTorch and calls the library's entry points for both
directions; without a gradient to compute they are the inference calls too.

A backward pass can be captured into a graph as any of PyTorch's: after warm-up
passes on a side stream, and with no eager graph over the same parameters still
alive (an output of an earlier pass that is kept holds one), since PyTorch would
add the captured gradients up on that graph's stream.

``kda_chunk`` allocates the outputs and workspaces with PyTorch and calls the
library's ``kda_fwd`` in the forward and ``kda_bwd`` in the backward; it adds
no arithmetic of its own.  Gradients flow to q, k, v, raw_gate, raw_beta,
A_log, dt_bias and initial_state from the output and from the final state.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import (FLAG_COMPLEMENT, FLAG_GATE_GIVEN, FLAG_INTERLEAVED, FLAG_KEEP_RECORDS, FLAG_NO_QK_NORM,
               FLAG_REUSE_RECORDS, FLAG_RMS_NORM, FLAG_SILU, FLAG_ZERO_REST, kda_bwd_ex, kda_bwd_workspace_size, kda_conv_bwd,
               kda_conv_bwd_workspace_size, kda_conv_fwd, kda_fwd_ex, kda_glr_bwd, kda_glr_bwd_workspace_size,
               kda_glr_fwd, kda_glr_states_size, kda_glr_workspace_size, kda_qk_rope_bwd,
               kda_qk_rope_bwd_workspace_size, kda_qk_rope_fwd, kda_workspace_size)

__all__ = ["kda_chunk", "kda_glr", "kda_short_conv", "kda_qk_norm_rope"]


def _sizes(q, v, cu_seqlens):
    B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    return B, T, H, K, V, N


def _as_taken(g, dtype):
    """A gradient as the kernels load it: of their type, contiguous and on a 16-byte boundary (a
    contiguous one need not be: the gradient of a piece of a ``cat`` is a view at the piece's offset)."""
    g = g.to(dtype).contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class _KdaChunk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, raw_gate, raw_beta, A_log, dt_bias, initial_state, scale, lower_bound,
                cu_seqlens, reuse_records, variant):
        B, T, H, K, V, N = _sizes(q, v, cu_seqlens)
        out = torch.empty_like(v)
        final_state = torch.empty(N, H, K, V, dtype=torch.float32, device=q.device)
        size = kda_bwd_workspace_size(B * T, H, N) if reuse_records else kda_workspace_size(B * T, H, N)
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device=q.device)
        kda_fwd_ex(q, k, v, raw_gate, raw_beta, scale, out, ws, A_log, dt_bias, lower_bound, initial_state,
                   final_state, cu_seqlens, flags=variant | (FLAG_KEEP_RECORDS if reuse_records else 0))
        ctx.save_for_backward(q, k, v, raw_gate, raw_beta, A_log, dt_bias, initial_state, cu_seqlens)
        ctx.scale, ctx.lower_bound, ctx.variant = scale, lower_bound, variant
        # the backward workspace starts with the forward's layout: keep it, records included
        ctx.ws = ws if reuse_records else None
        ctx.set_materialize_grads(False)
        return out, final_state

    @staticmethod
    def backward(ctx, d_out, d_final):
        q, k, v, raw_gate, raw_beta, A_log, dt_bias, initial_state, cu_seqlens = ctx.saved_tensors
        B, T, H, K, V, N = _sizes(q, v, cu_seqlens)
        d_out = torch.zeros_like(v) if d_out is None else _as_taken(d_out, torch.bfloat16)
        d_final = None if d_final is None else _as_taken(d_final, torch.float32)
        dq, dk, draw_gate = torch.empty_like(q), torch.empty_like(k), torch.empty_like(raw_gate)
        dv, draw_beta = torch.empty_like(v), torch.empty_like(raw_beta)
        dA_log, ddt_bias = torch.empty_like(A_log), torch.empty_like(dt_bias)
        dinit = None if initial_state is None else torch.empty_like(initial_state)
        if ctx.ws is not None:
            ws, flags = ctx.ws, FLAG_REUSE_RECORDS
        else:
            ws, flags = torch.empty(max(kda_bwd_workspace_size(B * T, H, N), 1), dtype=torch.uint8,
                                    device=q.device), 0
        kda_bwd_ex(q, k, v, raw_gate, raw_beta, ctx.scale, d_out, dq, dk, dv, draw_gate, draw_beta, dA_log,
                   ddt_bias, ws, A_log, dt_bias, ctx.lower_bound, initial_state=initial_state, d_final=d_final,
                   d_initial_state=dinit, cu_seqlens=cu_seqlens, flags=flags | ctx.variant)
        ctx.ws = None
        return dq, dk, dv, draw_gate, draw_beta, dA_log, ddt_bias, dinit, None, None, None, None, None


def kda_chunk(q, k, v, raw_gate, raw_beta, A_log, dt_bias, *, scale=None, lower_bound=-5.0,
              initial_state=None, cu_seqlens=None, reuse_records=False, qk_normalized=False):
    """Differentiable KDA forward; returns (out bf16 [B,T,H,V], final_state fp32 [N,H,K,V]).

    Inputs as for ``kda_fwd``: q, k, v, raw_gate bf16 [B,T,H,*]; raw_beta bf16 [B,T,H];
    A_log fp32 [H]; dt_bias fp32 [H,K]; initial_state fp32 [N,H,K,V] or None (zeros);
    cu_seqlens int32 [N+1] on the device (with B = 1) or None.  ``scale`` defaults to
    K^-1/2.  All tensors must be contiguous and on one GPU, and must not be modified in
    place between the forward and the backward.

    ``reuse_records`` runs the forward in a backward-sized workspace and keeps it until
    the backward, which then skips rebuilding the chunk records (KDA_FLAG_REUSE_RECORDS).
    It trades memory for time: the workspace (about 0.35 MB per chunk and head, 17 GB at
    T = 32768, H = 96) stays allocated from the forward to the backward, which uses the
    records up (a second backward would need the forward again).

    ``qk_normalized`` takes q and k as they are (KDA_FLAG_NO_QK_NORM), for rows that already have
    norm 1, as ``kda_qk_norm_rope`` makes with "l2" and no weights.  That they do is not checked here
    (``kda_fwd_ex`` records it in its workspace's fault word); longer rows give wrong results.
    Without it each row is normed here, also one that was scaled before, whose scale is lost.
    """
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return _KdaChunk.apply(q, k, v, raw_gate, raw_beta, A_log, dt_bias, initial_state, float(scale),
                           float(lower_bound), cu_seqlens, bool(reuse_records),
                           FLAG_NO_QK_NORM if qk_normalized else 0)


def _scratch(size, like):
    return torch.empty(max(size, 1), dtype=torch.uint8, device=like.device)


def _grad(g, like):
    """The gradient of an output of ``like``'s shape and type, zeros where there is none."""
    return torch.zeros_like(like, memory_format=torch.contiguous_format) if g is None else _as_taken(g, like.dtype)


def _count(x, cu_seqlens):
    return x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1


def _glr_forward(x, raw_gate, A_log, dt_bias, initial_state, lower_bound, cu_seqlens, flags, train):
    B, T, H, K = x.shape
    out = torch.empty_like(x)
    final = torch.empty(_count(x, cu_seqlens), H, K, dtype=torch.float32, device=x.device)
    states = _scratch(kda_glr_states_size(B * T, H, K), x) if train else None
    kda_glr_fwd(x, raw_gate, out, _scratch(kda_glr_workspace_size(B * T, H, K), x), A_log, dt_bias, lower_bound,
                initial_state, final, states, cu_seqlens, flags)
    return out, final, states


class _Glr(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, raw_gate, A_log, dt_bias, initial_state, lower_bound, cu_seqlens, flags):
        out, final, states = _glr_forward(x, raw_gate, A_log, dt_bias, initial_state, lower_bound, cu_seqlens, flags,
                                          True)
        ctx.save_for_backward(x, raw_gate, A_log, dt_bias, initial_state, cu_seqlens, states)
        ctx.lower_bound, ctx.flags = lower_bound, flags
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_final):
        x, raw_gate, A_log, dt_bias, initial_state, cu_seqlens, states = ctx.saved_tensors
        B, T, H, K = x.shape
        d_out = _grad(d_out, x)
        d_final = None if d_final is None else _as_taken(d_final, torch.float32)
        dx, dg = torch.empty_like(x), torch.empty_like(raw_gate)
        dA, dd = (None if t is None else torch.empty_like(t) for t in (A_log, dt_bias))
        di = None if initial_state is None else torch.empty_like(initial_state)
        kda_glr_bwd(x, raw_gate, states, d_out, dx, dg, dA, dd,
                    _scratch(kda_glr_bwd_workspace_size(B * T, H, K), x), A_log, dt_bias, ctx.lower_bound,
                    initial_state, d_final, di, cu_seqlens, ctx.flags)
        return dx, dg, dA, dd, di, None, None, None


def _wants_derivative(*tensors):
    """Whether the call has to be seen by autograd: an input requires a gradient, or carries a tangent
    (forward mode, which these operators do not have: autograd says so)."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def kda_glr(x, raw_gate, A_log=None, dt_bias=None, *, lower_bound=-5.0, initial_state=None, cu_seqlens=None,
            gate_given=False, complement=False):
    """Differentiable gated linear recurrence h_t = a_t h_{t-1} + b_t x_t; returns (h of x's type
    [B,T,H,K], final_state fp32 [N,H,K]).

    a_t = exp(g_t) with g_t = lower_bound sigmoid(exp(A_log) (raw_gate_t + dt_bias)), or raw_gate_t
    itself with ``gate_given`` (A_log and dt_bias must then be None); b_t = 1, or 1 - a_t with ``complement``.  x and
    raw_gate bf16 or fp32 [B,T,H,K]; A_log fp32 [H]; dt_bias fp32 [H,K]; initial_state fp32
    [N,H,K] or None; cu_seqlens int32 [N+1] (with B = 1) or None; rows behind the last sequence
    come back as zeros.  All tensors contiguous, on one GPU, and unchanged until the backward; x and
    raw_gate on a boundary of 4 elements, dt_bias and initial_state of 16 bytes, as PyTorch allocates
    (a view into a flat buffer may start elsewhere; the call then raises KdaError).
    """
    if gate_given and (A_log is not None or dt_bias is not None):
        raise ValueError("with gate_given there is no A_log and no dt_bias")
    flags = (FLAG_GATE_GIVEN if gate_given else 0) | (FLAG_COMPLEMENT if complement else 0) | FLAG_ZERO_REST
    args = (x, raw_gate, A_log, dt_bias, initial_state, float(lower_bound), cu_seqlens, flags)
    if _wants_derivative(x, raw_gate, A_log, dt_bias, initial_state):
        return _Glr.apply(*args)
    return _glr_forward(*args, False)[:2]


def _conv_forward(x, weight, bias, initial_state, cu_seqlens, flags):
    out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    final = torch.empty(_count(x, cu_seqlens), weight.shape[1] - 1, x.shape[2], dtype=x.dtype, device=x.device)
    kda_conv_fwd(x, weight, out, bias, initial_state, final, cu_seqlens, flags)
    return out, final


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, flags):
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.flags = flags
        ctx.set_materialize_grads(False)
        return _conv_forward(x, weight, bias, initial_state, cu_seqlens, flags)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, d_final):
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        d_out = _grad(d_out, x)
        d_final = None if d_final is None else _as_taken(d_final, x.dtype)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty_like(weight)
        db, di = (None if t is None else torch.empty_like(t) for t in (bias, initial_state))
        ws = _scratch(kda_conv_bwd_workspace_size(x.shape[0] * x.shape[1], x.shape[2], weight.shape[1]), x)
        kda_conv_bwd(x, weight, d_out, dx, dw, ws, bias, db, initial_state, d_final, di, cu_seqlens, ctx.flags)
        return dx, dw, db, di, None, None


def kda_short_conv(x, weight, bias=None, *, silu=True, initial_state=None, cu_seqlens=None):
    """Differentiable short causal depthwise convolution, with SiLU unless ``silu`` is False; returns
    (out [B,T,C], final_state [N,W-1,C]), both of x's type.

    x bf16 or fp32 [B,T,C], its tokens evenly apart (a slice of a wider projection's output will
    do); weight fp32 [C,W], W 2 to 4; bias fp32 [C] or None; initial_state [N,W-1,C] of x's type
    (the inputs before the first token, in order) or None for zeros; cu_seqlens int32 [N+1] (with
    B = 1) or None; rows behind the last sequence come back as zeros.  The final state is the next
    call's initial state.  x and initial_state start on a boundary of 4 elements, weight and bias of 16
    bytes (a view into a flat buffer that does not makes the call raise KdaError).
    """
    args = (x, weight, bias, initial_state, cu_seqlens, (FLAG_SILU if silu else 0) | FLAG_ZERO_REST)
    return _Conv.apply(*args) if _wants_derivative(x, weight, bias, initial_state) else _conv_forward(*args)


def _qk_forward(q, k, q_weight, k_weight, positions, inv_freq, eps, flags):
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    kda_qk_rope_fwd(q, k, q_out, k_out, positions, inv_freq, eps, q_weight, k_weight, flags)
    return q_out, k_out


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, flags):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.eps, ctx.flags = eps, flags
        ctx.set_materialize_grads(False)
        return _qk_forward(q, k, q_weight, k_weight, positions, inv_freq, eps, flags)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_q_out, d_k_out):
        q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
        dq, dk = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
        dqw, dkw = (None if t is None else torch.empty_like(t) for t in (q_weight, k_weight))
        ws = None
        if dqw is not None or dkw is not None:
            B, T, Hq, D = q.shape
            ws = _scratch(kda_qk_rope_bwd_workspace_size(B * T, Hq, k.shape[2], D), q)
        kda_qk_rope_bwd(q, k, _grad(d_q_out, q), _grad(d_k_out, k), dq, dk, positions, inv_freq, ctx.eps, q_weight,
                        k_weight, dqw, dkw, ws, ctx.flags)
        return dq, dk, dqw, dkw, None, None, None, None


_NORM = {"l2": 0, "rms": FLAG_RMS_NORM, "none": FLAG_NO_QK_NORM}


def kda_qk_norm_rope(q, k, positions=None, inv_freq=None, *, q_weight=None, k_weight=None, norm="l2", eps=1e-6,
                     interleaved=False):
    """Differentiable norm of queries and keys per head with the position rotation in the same pass;
    returns (q_out, k_out), contiguous, of the inputs' type.

    q [B,T,Hq,D], k [B,T,Hk,D] bf16 or fp32, tokens and heads evenly apart (slices of one
    projection's output will do); ``norm`` "l2" (x / sqrt(sum x^2 + eps), the core's), "rms"
    (x / sqrt(mean x^2 + eps)) or "none"; q_weight, k_weight fp32 [D] or None; positions int32
    [B,T] and inv_freq fp64 [R/2] (radians per position) turn the pairs (i, i + R/2) of the first
    R channels, or (2i, 2i + 1) with ``interleaved``; None leaves them.  inv_freq is not
    differentiated: one that requires a gradient is refused.  q and k start on a boundary of 4
    elements, and so do their rows.

    With "l2" and no weights the results are unit rows, as ``kda_chunk`` takes them with
    ``qk_normalized`` and ``kda_fwd_ex`` with FLAG_NO_QK_NORM.  Rows with weights or of "rms" are for
    layers without a norm of their own: the core's takes their scale off again.
    """
    if norm not in _NORM:
        raise ValueError(f"norm must be one of {sorted(_NORM)}")
    if inv_freq is not None and inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq has no gradient here: pass inv_freq.detach()")
    args = (q, k, q_weight, k_weight, positions, inv_freq, float(eps),
            _NORM[norm] | (FLAG_INTERLEAVED if interleaved else 0))
    return _QkNormRope.apply(*args) if _wants_derivative(q, k, q_weight, k_weight, inv_freq) else _qk_forward(*args)
