"""The token mixers on the GPU as a model uses them, one after another in a stack, and over arrays
that 32-bit offsets do not reach.  Tolerances are those of the operators' own tests, step by step:
every operator is held to its formula at the inputs and gradients that it was given."""

import numpy as np
import pytest
import torch

import chunked_gated_delta_amd as kda
import test_gpu_attn as at
import test_gpu_linear_attn as la
from chunked_gated_delta_amd.function import kda_attn, kda_chunk, kda_linear_attn, kda_qk_norm_rope
from test_gpu_around import DEV, Rand, near, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("lengths", [None, [70, 0, 1, 128, 201]])
def test_layers_of_every_kind_after_each_other(lengths):
    """One residual stream of heads: linear attention, the core, causal attention with shared key heads, all
    of them over the same packed prompts, queries and keys normed and turned before each."""
    say("stack", lengths)
    r = Rand(400)
    T, H, Hk, D = 400, 4, 2, 128
    cu = None if lengths is None else torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32)
    pos = torch.arange(T, dtype=torch.int32)[None] if cu is None else torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths])[None]
    pos, dcu = pos.to(DEV), None if cu is None else cu.to(DEV)
    freq = torch.logspace(0, -3, D // 2, dtype=torch.float64, device=DEV)
    wide = r(1, T, 3 * H + 2 * Hk, D, dtype=BF).to(DEV).requires_grad_()
    g = (-torch.exp(r(H) - 3.0)).to(DEV).requires_grad_()
    gate, beta = r(1, T, H, D, dtype=BF).to(DEV), r(1, T, H, dtype=BF).to(DEV)
    A_log, bias = r(H).to(DEV), r(H, D).to(DEV)
    keep = lambda *ts: [t.retain_grad() for t in ts]  # noqa: E731

    q1, k1 = kda_qk_norm_rope(wide[:, :, :H], wide[:, :, H:2 * H], pos, freq)
    v1 = wide[:, :, 2 * H:3 * H]
    o1, s1 = kda_linear_attn(q1, k1, v1, g, cu_seqlens=dcu)
    o2, _ = kda_chunk(q1, k1, o1, gate, beta, A_log, bias, cu_seqlens=dcu, qk_normalized=True)
    q3, k3 = kda_qk_norm_rope(o2, wide[:, :, 3 * H:3 * H + Hk], pos, freq, norm="rms")
    v3 = wide[:, :, 3 * H + Hk:]
    o3, lse = kda_attn(q3, k3, v3, cu_seqlens=dcu)
    keep(q1, k1, v1, o1, s1, q3, k3, v3)
    d3, dl, ds = r(*o3.shape, dtype=BF), r(*lse.shape), r(*s1.shape)
    ((o3.float() * d3.to(DEV).float()).sum() + (lse * dl.to(DEV)).sum() + (s1 * ds.to(DEV)).sum()).backward()

    cpu = lambda t: t.detach().cpu()  # noqa: E731
    c = dict(q=cpu(q3), k=cpu(k3), v=cpu(v3), cq=cu, ck=cu, d_out=d3, d_lse=dl, scale=D ** -0.5, rest=0)
    val, tol = at.expected(c)
    for n, t in dict(out=o3, lse=lse, dq=q3.grad, dk=k3.grad, dv=v3.grad).items():
        near("attention " + n, t.flatten(0, 1), val[n], tol[n])

    c = dict(q=cpu(q1), k=cpu(k1), v=cpu(v1), g=cpu(g), init=None, cu=cu, d_out=cpu(o1.grad), d_fin=ds, scale=D ** -0.5)
    (out, fin), grads = la.oracle(c)
    t_out, t_grad = la.tolerances(c, la.oracle(c, absolute=True))
    near("linear attention out", o1.flatten(0, 1), out, HALF * out.abs() + t_out[0])
    near("linear attention state", s1, fin, t_out[1])
    near("linear attention dv", v1.grad.flatten(0, 1), *(x.flatten(0, 1) for x in (grads[2], HALF * grads[2].abs() + t_grad[2])))
    near("linear attention d_log_decay", g.grad, grads[3], t_grad[3])
    # q1 and k1 get two gradients, of the core's too: those of the linear attention by itself
    leaves = [t.detach().requires_grad_() for t in (q1, k1)]
    o, s = kda_linear_attn(*leaves, v1.detach(), g.detach(), cu_seqlens=dcu)
    got = torch.autograd.grad([o, s], leaves, [o1.grad, ds.to(DEV)])
    assert torch.equal(o, o1) and torch.equal(s, s1)
    for n, t, want, size in zip(("dq", "dk"), got, grads, t_grad):
        near("linear attention " + n, t.flatten(0, 1), want.flatten(0, 1), (HALF * want.abs() + size).flatten(0, 1))
    assert all(torch.isfinite(t.grad.float()).all() and t.grad.float().abs().max() > 0 for t in (wide, q1, k1))


def test_heads_before_tokens():
    """[H, T, D] arrays, seen as tokens and heads, give the bits of contiguous ones, gradients too."""
    r = Rand(401)
    T = 333
    for op, H in (("la", (5, 5, 5)), ("attn", (64, 1, 1)), ("attn", (6, 3, 3))):
        say(op, H)
        x = [r(1, h, T, 128, dtype=BF).to(DEV).requires_grad_() for h in H]
        y = [t.detach().transpose(1, 2).contiguous().requires_grad_() for t in x]
        d, e = r(1, T, H[0], 128, dtype=BF).to(DEV), torch.tensor([-0.1] * H[0], device=DEV)
        got = []
        for leaves, seen in ((x, [t.transpose(1, 2) for t in x]), (y, y)):
            out = (kda_linear_attn(*seen, e) if op == "la" else kda_attn(*seen))[0]
            got.append([out, *torch.autograd.grad(out, leaves, d)])
        assert torch.equal(got[0][0], got[1][0])
        assert all(torch.equal(a.transpose(1, 2), b) for a, b in zip(got[0][1:], got[1][1:]))


def test_hundreds_of_short_sequences():
    r = np.random.RandomState(402)
    lengths = [int(n) for n in r.randint(0, 9, 700)]
    say("linear attention")
    c = la.case(403, 1, 0, 2, 64, 64, lengths=lengths)
    (out, fin), grads = la.oracle(c)
    t_out, t_grad = la.tolerances(c, la.oracle(c, absolute=True))
    got, d = la.fwd(c), la.bwd(c)
    near("out", got[0].flatten(0, 1), out, HALF * out.abs() + t_out[0])
    near("final", got[1], fin, t_out[1])
    for n, x, want, tol in zip(("dq", "dk", "dv"), d, grads, t_grad):
        near(n, x.flatten(0, 1), want.flatten(0, 1), (HALF * want.abs() + tol).flatten(0, 1))
    near("d_log_decay", d[3], grads[3], t_grad[3])
    near("d_initial_state", d[4], grads[4], t_grad[4])
    say("attention")
    at.check(at.case(404, 1, 0, 2, 1, 64, lengths=lengths, pasts=[int(n) for n in r.randint(0, 9, 700)]))


def test_what_a_nan_reaches_in_the_backward():
    """Behind and before its token no more than the formula says, and the 127 tokens around it."""
    c = at.case(407, 1, 700, 4, 2)
    clean, where = at.bwd(c), 300
    b = dict(c, q=c["q"].clone())
    b["q"][0, where, 1] = float("nan")
    dq, dk, dv = at.bwd(b)
    others = torch.arange(700) != where
    assert torch.equal(dq[:, others], clean[0][:, others]) and torch.equal(dq[:, :, [0, 2, 3]], clean[0][:, :, [0, 2, 3]])
    for x, y in ((dk, clean[1]), (dv, clean[2])):
        assert torch.equal(x[:, where + 128:], y[:, where + 128:]) and torch.equal(x[:, :, 1], y[:, :, 1])
    b = dict(c, k=c["k"].clone())
    b["k"][0, where, 0] = float("nan")
    dq = at.bwd(b)[0]
    assert torch.equal(dq[:, :where - 127], clean[0][:, :where - 127]) and torch.equal(dq[:, :, 2:], clean[0][:, :, 2:])


def test_a_cache_of_more_than_two_to_the_31_elements():
    """A token behind 2.2 million earlier ones of eight heads, and its gradients.  Three keys, the first, a
    middle one and the last, outweigh the rest.  Sums of the forward run over a 64th of the keys."""
    r = Rand(405)
    H, D, n = 8, 128, (1 << 21) + 100003
    gen = torch.Generator(DEV).manual_seed(405)
    k, v = (torch.empty(1, n, H, D, dtype=BF, device=DEV) for _ in range(2))
    for t in (k, v):
        for i in range(0, n, 1 << 18):
            t[:, i:i + (1 << 18)] = torch.randn(t[:, i:i + (1 << 18)].shape, device=DEV, generator=gen).to(BF)
    assert k.numel() > 1 << 31
    q = r(1, 1, H, D, dtype=BF).to(DEV)
    for i in (0, n // 2 + 7, n - 1):
        k[:, i] = q[:, 0]
    d_out, d_lse, scale = r(1, 1, H, D, dtype=BF).to(DEV), r(1, 1, H).to(DEV), 0.15
    out, lo, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(1, 1, H, device=DEV)
    ws = torch.empty(kda.kda_attn_workspace_size(1, n, H, H, D, 1), dtype=torch.uint8, device=DEV)
    kda.kda_attn_fwd(q, k, v, scale, out, lse, ws, lo)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(kda.kda_attn_bwd_workspace_size(1, n, H, H, D, 1), dtype=torch.uint8, device=DEV)
    kda.kda_attn_bwd(q, k, v, scale, out, lo, lse, d_out, dq, dk, dv, ws, d_lse)
    for h in range(H):
        x, y, w, d = (t[0, :, h].double() for t in (q, k, v, d_out))
        s = scale * (x @ y.T)[0]
        want = torch.logsumexp(s, 0)
        p = torch.exp(s - want)
        off = (130 * 2.0 ** -24 * scale * (x.abs() @ y.abs().T)).amax() * 2 + 2.0 ** -20
        many = (n // 64 + 64) * 2.0 ** -24
        o, size = p @ w, p @ w.abs()
        near("out", out[0, 0, h], o.cpu(), ((HALF + off + many) * size * (1 + HALF) + HALF * o.abs()).cpu())
        near("lse", lse[0, 0, h], want.cpu(), (off + many + 2.0 ** -22 * (1 + want.abs())).cpu())
        dp, e = (d @ w.T)[0], d_lse[0, 0, h].double()
        gd = (d[0] * o).sum() - e
        ds = p * (dp - gd)
        dsz = p * (128 * 2.0 ** -24 * (d.abs() @ w.abs().T)[0] + (HALF + off + many + 2.0 ** -15) * (d.abs()[0] * size).sum()
                   + 2.0 ** -22 * e.abs()) + (off + HALF + many) * ds.abs()
        for name, got, want, tol in (
                ("dq", dq[0, 0, h], scale * ds @ y, scale * dsz @ y.abs() + n * 2.0 ** -24 * scale * ds.abs() @ y.abs()),
                *((name, t[0, rows, h], val[rows], tol[rows])
                  for name, t, val, tol in (("dk", dk, scale * ds[:, None] * x, scale * (dsz + 2.0 ** -24 * ds.abs())[:, None] * x.abs()),
                                            ("dv", dv, p[:, None] * d, (p * (off + HALF + 2.0 ** -24))[:, None] * d.abs()))
                  for rows in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)))):
            near(name, got, want.cpu(), (tol * (1 + HALF) + HALF * want.abs() + 1e-30).cpu())


def test_linear_attention_over_more_than_two_to_the_31_elements():
    """Rows at the arrays' ends, against the formula over those rows and the state that reaches them: of what
    is 4096 tokens away the decays, e^-0.05 a token or less, leave e^-204."""
    H, D, T, n = 16, 64, (1 << 21) + 37, 1037
    gen = torch.Generator(DEV).manual_seed(406)
    q, k, v, d = (torch.empty(1, T, H, D, dtype=BF, device=DEV) for _ in range(4))
    for t in (q, k, v, d):
        for i in range(0, T, 1 << 18):
            t[:, i:i + (1 << 18)] = torch.randn(t[:, i:i + (1 << 18)].shape, device=DEV, generator=gen).to(BF)
    assert q.numel() > 1 << 31
    r = Rand(406)
    g, d_fin, scale = -0.05 - r(H).abs(), r(1, H, D, D), D ** -0.5
    out, fin = torch.empty_like(v), torch.empty(1, H, D, D, device=DEV)
    ws = torch.empty(kda.kda_la_bwd_workspace_size(T, H, D, D, 1), dtype=torch.uint8, device=DEV)
    kda.kda_la_fwd(q, k, v, g.to(DEV), scale, out, ws, None, fin)
    grads = [torch.empty_like(q) for _ in range(3)]
    kda.kda_la_bwd(q, k, v, g.to(DEV), scale, d, *grads, ws, torch.empty(H, device=DEV), None, d_fin.to(DEV))
    far = 4096
    for a, z, behind in ((0, n, 0), (T - n - far, T, far)):  # rows behind the first 4096 of the last part are held to it
        part = {name: t[:, a:z].cpu() for name, t in zip(("q", "k", "v", "d_out"), (q, k, v, d))}
        # behind the first rows comes a gradient of their state, which is not known here: only what it does not reach
        c = dict(part, g=g, init=None, cu=None, d_fin=d_fin if z == T else torch.zeros_like(d_fin), scale=scale)
        (o, s), dd = la.oracle(c)
        t_out, t_grad = la.tolerances(c, la.oracle(c, absolute=True))
        live = slice(behind, z - a)
        say("rows", a, z)
        near("out", out[0, a:z][live], o[live], (HALF * o.abs() + t_out[0])[live])
        names = ("dq", "dk", "dv") if z == T else ("dq",)
        for name, got, want, tol in zip(names, grads, dd, t_grad):
            near(name, got[0, a:z][live], want[0][live], (HALF * want.abs() + tol)[0][live])
    near("final", fin, s, t_out[1])
