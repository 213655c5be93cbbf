"""fp64 oracles of the token mixers beside the core: linear attention with a decay for each head, and
causal attention with grouped heads.

Test infrastructure only; see the package docstring.  Both are written pair by pair, from the sums
over the tokens that each token sees, with differentiable PyTorch CPU operations in fp64; the tests
pin them by token-by-token forms, closed forms and central finite differences.
"""

from __future__ import annotations

import torch

from .around import bounds


def linear_attn(q, k, v, log_decay, initial_state=None, cu_seqlens=None, scale=1.0):
    """fp64 tensors in, (out [B*T, H, V], final [N, H, K, V]) out; rows of no sequence are zero."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    q, k, v = (x.flatten(0, 1).transpose(0, 1) for x in (q, k, v))
    a = log_decay.exp()[:, None, None]
    out, finals, at = [], [], 0
    for n, (lo, hi) in enumerate(bounds(B, T, cu_seqlens)):
        s0 = torch.zeros(H, K, V, dtype=torch.float64) if initial_state is None else initial_state[n]
        t = torch.arange(hi - lo, dtype=torch.float64)
        gap = (t[:, None] - t).clamp(min=0)
        pairs = (q[:, lo:hi] @ k[:, lo:hi].transpose(1, 2)) * (a ** gap).tril()
        out.append(scale * (pairs @ v[:, lo:hi] + a ** (t[:, None] + 1) * (q[:, lo:hi] @ s0)))
        finals.append((k[:, lo:hi] * a ** (hi - lo - 1 - t[:, None])).transpose(1, 2) @ v[:, lo:hi] + a ** (hi - lo) * s0)
        at = hi
    out.append(torch.zeros(H, B * T - at, V, dtype=torch.float64))
    return torch.cat(out, 1).transpose(0, 1), torch.stack(finals)


def attn(q, k, v, scale, cu_q=None, cu_k=None):
    """fp64 q [B, Tq, Hq, D], k, v [B, Tk, Hk, D] in, (out [B*Tq, Hq, D], lse [B*Tq, Hq]) out.  Query i of
    a sequence of nq queries and nk keys sees the keys up to i + nk - nq; one that sees none gives
    zeros and minus infinity, as do rows of no sequence."""
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    q, k, v = (x.flatten(0, 1).transpose(0, 1) for x in (q, k, v))
    k, v = (x.repeat_interleave(Hq // Hk, 0) for x in (k, v))
    outs, sums = [], []
    at = 0
    for (lo, hi), (a, z) in zip(bounds(B, Tq, cu_q), bounds(B, Tk, cu_q if cu_k is None else cu_k)):
        nq, nk = hi - lo, z - a
        sees = torch.arange(nk)[None] <= torch.arange(nq)[:, None] + (nk - nq)
        some = sees.any(1)
        score = scale * (q[:, lo:hi] @ k[:, a:z].transpose(1, 2))
        score = torch.where(sees, score, torch.full_like(score, -torch.inf))
        score = torch.where(some[:, None], score, torch.zeros_like(score))  # rows without keys: no NaN to differentiate
        s = torch.logsumexp(score, -1) if nk else torch.zeros(Hq, nq, dtype=torch.float64)
        p = torch.exp(score - s[..., None]) * sees
        outs.append(p @ v[:, a:z])
        sums.append(torch.where(some, s, torch.full_like(s, -torch.inf)))
        at = hi
    outs.append(torch.zeros(Hq, B * Tq - at, D, dtype=torch.float64))
    sums.append(torch.full((Hq, B * Tq - at), -torch.inf, dtype=torch.float64))
    return torch.cat(outs, 1).transpose(0, 1), torch.cat(sums, 1).transpose(0, 1)
