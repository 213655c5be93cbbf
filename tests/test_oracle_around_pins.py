"""Pins of the fp64 oracles of the operators around the core (oracle/around.py), on the CPU:
closed forms, packed runs against separate ones, and gradients against central differences."""

import math

import pytest
import torch

from oracle import around as A

F = torch.float64


def rand(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=F) * std


def differences(f, leaves, cots, live, eps=1e-5, tries=6):
    """Directional central differences of the loss against the gradients, one leaf at a time."""
    outs, g = A.grads(f, leaves, cots)
    for i in live:
        for s in range(tries):
            d = rand(*leaves[i].shape, seed=100 + 7 * s + i)

            def loss(e):
                at = [t if t is None else A.f64(t) for t in leaves]
                at[i] = at[i] + e * d
                o = f(*at)
                o = o if isinstance(o, tuple) else (o,)
                return sum((a * c.reshape(a.shape)).sum() for a, c in zip(o, cots) if c is not None).item()

            num, ana = (loss(eps) - loss(-eps)) / (2 * eps), (g[i] * d).sum().item()
            # truncation eps^2 and fp64 rounding / eps, both relative to the sums' size
            assert abs(num - ana) <= 1e-7 * (1 + abs(ana) + d.norm().item() * g[i].norm().item()), (i, s, num, ana)
    return outs, g


def test_glr_closed_forms():
    x, T = rand(1, 9, 2, 4), 9
    # decay zero dropped: g = 0 sums the inputs; g = -inf forgets
    out, fin = A.glr(x, torch.zeros(1, T, 2, 4, dtype=F), None, None, -5.0, given=True)
    assert torch.allclose(out, x[0].cumsum(0), atol=1e-14) and torch.equal(fin[0], out[-1])
    out, _ = A.glr(x, torch.full((1, T, 2, 4), -math.inf, dtype=F), None, None, -5.0, given=True)
    assert torch.equal(out, x[0])
    # constant decay a and input 1 scaled by 1 - a: 1 - a^t from zero
    a = 0.7
    out, _ = A.glr(torch.ones(1, T, 2, 4, dtype=F), torch.full((1, T, 2, 4), math.log(a), dtype=F), None, None, -5.0,
                   given=True, complement=True)
    want = 1 - a ** torch.arange(1, T + 1, dtype=F)
    assert torch.allclose(out, want[:, None, None].expand(T, 2, 4), atol=1e-13)
    # the gate: raw far up gives lower_bound, far down 0
    out, _ = A.glr(x, torch.full((1, T, 2, 4), 1e4, dtype=F), torch.zeros(2, dtype=F), torch.zeros(2, 4, dtype=F), -2.0)
    assert torch.allclose(out[1], x[0, 1] + math.exp(-2.0) * x[0, 0], atol=1e-14)


def test_packed_equals_separate():
    cu = [0, 4, 4, 5, 11]
    x, g, init = rand(1, 12, 2, 4, seed=1), rand(1, 12, 2, 4, seed=2), rand(4, 2, 4, seed=3)
    al, dt = rand(2, seed=4), rand(2, 4, seed=5)
    out, fin = A.glr(x, g, al, dt, -5.0, init, cu, complement=True)
    w, b, ci = rand(8, 3, seed=6), rand(8, seed=7), rand(4, 2, 8, seed=8)
    xc = x.reshape(1, 12, 8)
    co, cf = A.conv(xc, w, b, ci, cu)
    for n in range(4):
        lo, hi = cu[n], cu[n + 1]
        o, f = A.glr(x[:, lo:hi], g[:, lo:hi], al, dt, -5.0, init[n:n + 1], complement=True)
        assert torch.equal(out[lo:hi], o) and torch.equal(fin[n], f[0])
        o, f = A.conv(xc[:, lo:hi], w, b, ci[n:n + 1])
        assert torch.equal(co[lo:hi], o) and torch.equal(cf[n], f[0])
    assert not out[11:].any() and not co[11:].any()


def test_conv_closed_forms():
    x = rand(2, 10, 8, seed=1)
    w = torch.zeros(8, 4, dtype=F)
    w[:, 1] = 1.0  # picks the input two rows back
    out, fin = A.conv(x, w, silu=False)
    assert torch.equal(out.reshape(2, 10, 8)[:, 2:], x[:, :-2]) and torch.equal(fin, x[:, -3:])
    ref = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)), rand(8, 1, 4, seed=2),
                                     rand(8, seed=3), groups=8).transpose(1, 2)
    out, _ = A.conv(x, rand(8, 1, 4, seed=2)[:, 0], rand(8, seed=3))
    assert torch.allclose(out.reshape(2, 10, 8), torch.nn.functional.silu(ref), atol=1e-13)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_closed_forms(inter):
    x = rand(1, 5, 2, 16, seed=1)
    pos = torch.tensor([[0, 1, 7, 100, -3]])
    f = torch.tensor([1.0, 0.3, 0.01, math.pi], dtype=F)
    y = A.qk_norm_rope(x, pos, f, interleaved=inter)
    # a rotation keeps the norm: unit rows; position 0 turns nothing; the tail stays
    assert torch.allclose(y.square().sum(-1), torch.ones(1, 5, 2, dtype=F), atol=1e-5)
    n = A.qk_norm_rope(x, None, None)
    assert torch.allclose(y[:, 0], n[:, 0]) and torch.equal(y[..., 8:], n[..., 8:])
    # scores depend on the distance alone
    q, k = rand(1, 1, 1, 16, seed=2), rand(1, 1, 1, 16, seed=3)
    at = lambda t, p: A.qk_norm_rope(t, torch.tensor([[p]]), f, interleaved=inter)  # noqa: E731
    assert torch.allclose((at(q, 9) * at(k, 4)).sum(), (at(q, 105) * at(k, 100)).sum(), atol=1e-10)
    # one pair by hand
    i, j = (0, 1) if inter else (0, 4)
    c, s = math.cos(7.0), math.sin(7.0)
    assert torch.allclose(y[0, 2, 0, i], n[0, 2, 0, i] * c - n[0, 2, 0, j] * s)
    assert torch.allclose(y[0, 2, 0, j], n[0, 2, 0, j] * c + n[0, 2, 0, i] * s)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("complement", [False, True])
def test_glr_gradients_by_differences(given, complement):
    cu = [0, 3, 3, 7]
    x, g = rand(1, 7, 2, 4, seed=1), rand(1, 7, 2, 4, seed=2)
    leaves = [x, -g.abs() if given else g, None if given else rand(2, seed=3), None if given else rand(2, 4, seed=4),
              rand(3, 2, 4, seed=5)]
    differences(lambda x, g, al, dt, i: A.glr(x, g, al, dt, -5.0, i, cu, given, complement), leaves,
                [rand(7, 2, 4, seed=6), rand(3, 2, 4, seed=7)], [0, 1, 4] if given else [0, 1, 2, 3, 4])


@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradients_by_differences(silu):
    cu = [0, 2, 2, 8]
    differences(lambda x, w, b, i: A.conv(x, w, b, i, cu, silu),
                [rand(1, 8, 8, seed=1), rand(8, 4, seed=2), rand(8, seed=3), rand(3, 3, 8, seed=4)],
                [rand(8, 8, seed=5), rand(3, 3, 8, seed=6)], [0, 1, 2, 3])


@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradients_by_differences(norm, inter):
    pos, f = torch.tensor([[5, 6, 7]]), torch.tensor([1.0, 0.2, 0.03, 0.004], dtype=F)
    differences(lambda x, w: A.qk_norm_rope(x, pos, f, w, norm, interleaved=inter),
                [rand(1, 3, 2, 16, seed=1), rand(16, seed=2)], [rand(1, 3, 2, 16, seed=3)], [0, 1])
