"""fp64 oracles of the operators around the core: gated linear recurrence, short causal
convolution, norm and rotation of queries and keys.

Test infrastructure only; see the package docstring.  Each is written token by token (or as a
complex product, for the rotation) from its definition with differentiable PyTorch CPU
operations in fp64, so that ``grads`` gives the exact gradients by autograd; the tests pin
those by central finite differences and the forwards by closed forms.
"""

from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


def bounds(B, T, cu_seqlens):
    """(first, end) rows of every sequence on the packed axis [B * T]."""
    if cu_seqlens is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    cu = [int(c) for c in cu_seqlens]
    return list(zip(cu[:-1], cu[1:]))


def glr(x, raw_gate, A_log, dt_bias, lower_bound, initial_state=None, cu_seqlens=None, given=False, complement=False):
    """fp64 tensors in, (out [B*T, H, K], final [N, H, K]) out; rows of no sequence are zero."""
    B, T, H, K = x.shape
    xf, gf = x.reshape(B * T, H, K), raw_gate.reshape(B * T, H, K)
    rows, finals = [torch.zeros(H, K, dtype=torch.float64)] * (B * T), []
    for n, (lo, hi) in enumerate(bounds(B, T, cu_seqlens)):
        h = torch.zeros(H, K, dtype=torch.float64) if initial_state is None else initial_state[n]
        for t in range(lo, hi):
            g = gf[t] if given else lower_bound * torch.sigmoid(A_log.exp()[:, None] * (gf[t] + dt_bias))
            a = g.exp()
            u = -torch.expm1(g) * xf[t] if complement else xf[t]
            h = a * h + u
            rows[t] = h
        finals.append(h)
    out = torch.stack(rows) if rows else torch.zeros(0, H, K, dtype=torch.float64)
    return out, torch.stack(finals)


def conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, silu=True):
    """fp64 tensors in, (out [B*T, C], final [N, W-1, C]) out; rows of no sequence are zero."""
    B, T, C = x.shape
    W = weight.shape[1]
    xf = x.reshape(B * T, C)
    rows, finals = [torch.zeros(C, dtype=torch.float64)] * (B * T), []
    for n, (lo, hi) in enumerate(bounds(B, T, cu_seqlens)):
        past = [torch.zeros(C, dtype=torch.float64)] * (W - 1) if initial_state is None else list(initial_state[n])
        for t in range(lo, hi):
            past.append(xf[t])
            z = sum(weight[:, j] * past[len(past) - W + j] for j in range(W))
            z = z if bias is None else z + bias
            rows[t] = z * torch.sigmoid(z) if silu else z
        finals.append(torch.stack(past[len(past) - (W - 1):]))
    out = torch.stack(rows) if rows else torch.zeros(0, C, dtype=torch.float64)
    return out, torch.stack(finals)


def qk_norm_rope(x, positions, inv_freq, weight=None, norm="l2", eps=1e-6, interleaved=False):
    """One of q and k: fp64 x [B, T, H, D] in, the same shape out."""
    D = x.shape[-1]
    y = x
    if norm != "none":
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / (D if norm == "rms" else 1) + eps)
    y = y if weight is None else y * weight
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    if R == 0:
        return y
    angle = positions.to(torch.float64)[:, :, None, None] * inv_freq
    head = y[..., :R]
    re, im = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :R // 2], head[..., R // 2:])
    pair = torch.complex(re.contiguous(), im.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    head = torch.stack([pair.real, pair.imag], -1).flatten(-2) if interleaved else torch.cat([pair.real, pair.imag], -1)
    return torch.cat([head, y[..., R:]], -1)


def grads(f, leaves, cotangents):
    """Outputs of f(*leaves), and the gradients of sum <cotangent, output> in every leaf that is one."""
    live = [None if t is None else f64(t).requires_grad_(True) for t in leaves]
    outs = f(*live)
    outs = outs if isinstance(outs, tuple) else (outs,)
    loss = sum((o * f64(c).reshape(o.shape)).sum() for o, c in zip(outs, cotangents) if c is not None)
    ask = [t for t in live if t is not None]
    got = iter(torch.autograd.grad(loss, ask, allow_unused=True))
    g = [None if t is None else next(got) for t in live]
    g = [torch.zeros_like(t) if t is not None and d is None else d for t, d in zip(live, g)]
    return [o.detach() for o in outs], g
