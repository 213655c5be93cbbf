"""Pins of the token mixers' fp64 oracles: token-by-token forms, closed forms, central differences."""

import math

import pytest
import torch

from oracle import around as A
from oracle import mixers as M

F64 = torch.float64


def rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=F64)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 11], [0, 9]])
def test_linear_attention_is_its_recurrence(cu):
    r = rand(1)
    B, T, H, K, V = 1, 11, 2, 3, 5
    q, k, v, g = r(B, T, H, K), r(B, T, H, K), r(B, T, H, V), -r(H).abs()
    N = 1 if cu is None else len(cu) - 1
    init = r(N, H, K, V)
    out, fin = M.linear_attn(q, k, v, g, init, cu, 0.7)
    want = torch.zeros_like(out)
    for n, (lo, hi) in enumerate(A.bounds(B, T, cu)):
        S = init[n]
        for t in range(lo, hi):
            S = g.exp()[:, None, None] * S + k[0, t][:, :, None] * v[0, t][:, None, :]
            want[t] = 0.7 * (S * q[0, t][:, :, None]).sum(1)
        assert torch.allclose(fin[n], S, rtol=1e-13, atol=1e-13)
    assert torch.allclose(out, want, rtol=1e-13, atol=1e-13)


def test_linear_attention_closed_forms():
    r = rand(2)
    q, k, v = r(1, 6, 1, 4), r(1, 6, 1, 4), r(1, 6, 1, 4)
    out, fin = M.linear_attn(q, k, v, torch.tensor([-math.inf], dtype=F64))
    assert torch.allclose(out[:, 0], (q * k).sum(-1)[0] * v[0, :, 0])  # nothing kept
    assert torch.allclose(fin[0, 0], torch.outer(k[0, 5, 0], v[0, 5, 0]))
    one = torch.ones(1, 6, 1, 1, dtype=F64)
    out, _ = M.linear_attn(one, one, one, torch.tensor([math.log(0.5)], dtype=F64))
    assert torch.allclose(out[:, 0, 0], 2 - 0.5 ** torch.arange(6, dtype=F64))  # 1 + 1/2 + 1/4 ...


def test_attention_closed_forms():
    r = rand(3)
    q, k, v = r(1, 5, 4, 3), r(1, 5, 2, 3), r(1, 5, 2, 3)
    out, lse = M.attn(torch.zeros_like(q), k, v, 1.0)  # equal scores: running means, log counts
    mean = v[0].cumsum(0) / torch.arange(1, 6, dtype=F64)[:, None, None]
    assert torch.allclose(out, mean.repeat_interleave(2, 1))
    assert torch.allclose(lse, torch.arange(1, 6, dtype=F64).log()[:, None].expand(5, 4))
    out, lse = M.attn(q, k, v, 0.5)
    assert torch.allclose(out[0], v[0, 0].repeat_interleave(2, 0))  # the first token sees itself
    for t in range(5):  # one query at a time behind its keys
        o, s = M.attn(q[:, t:t + 1], k[:, :t + 1], v[:, :t + 1], 0.5)
        assert torch.allclose(o[0], out[t]) and torch.allclose(s[0], lse[t])


def test_attention_rows_without_keys():
    r = rand(4)
    q, k, v = r(1, 7, 2, 3), r(1, 3, 1, 3), r(1, 3, 1, 3)
    out, lse = M.attn(q, k, v, 1.0, [0, 4, 6], [0, 2, 2])  # two queries before the keys; no key at all; no sequence
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all() and torch.isfinite(lse[2:4]).all()
    assert (out[4:] == 0).all() and (lse[4:] == -math.inf).all()
    _, g = A.grads(lambda q, k, v: M.attn(q, k, v, 1.0, [0, 4, 6], [0, 2, 2])[0], [q, k, v], [r(7, 2, 3)])
    assert all(torch.isfinite(t).all() for t in g) and (g[0][0, :2] == 0).all() and (g[1][0, 2] == 0).all()


@pytest.mark.parametrize("which", ["la", "attn"])
def test_gradients_are_differences(which):
    r = rand(5)
    if which == "la":
        leaves = [r(1, 9, 2, 3), r(1, 9, 2, 3), r(1, 9, 2, 4), -r(2).abs(), r(3, 2, 3, 4)]
        f = lambda *t: M.linear_attn(*t, [0, 4, 4, 9], 0.6)  # noqa: E731
        cot = [r(9, 2, 4), r(3, 2, 3, 4)]
    else:
        leaves = [r(1, 7, 4, 3), r(1, 9, 2, 3), r(1, 9, 2, 3)]
        f = lambda *t: M.attn(*t, 0.6, [0, 4, 7], [0, 5, 9])  # noqa: E731
        cot = [r(7, 4, 3), r(7, 4)]
    _, got = A.grads(f, leaves, cot)
    loss = lambda t: sum((o * c).sum() for o, c in zip(f(*t), cot))  # noqa: E731
    for i, x in enumerate(leaves):
        for _ in range(3):
            d, h = r(*x.shape), 1e-5
            up, down = ([y + s * d * h if j == i else y for j, y in enumerate(leaves)] for s in (1, -1))
            assert abs((loss(up) - loss(down)) / (2 * h) - (got[i] * d).sum()) <= 1e-7 * (1 + (got[i] * d).abs().sum())
