"""Causal attention with grouped heads on the GPU against its fp64 oracle (oracle/mixers.py).

Tolerances, element by element, from the oracle's own numbers.  Scores are sums of 128 exact products
in fp32 and enter an exponential: every weight is off by at most E = (130 2^-24) sum |q||k| scale +
2^-20 relative (the exponential and the log-sum included).  As MFMA operands weights and dS are rounded
to bf16 (half a step, 2^-8 of each at most: eps / 2), results too.  do.o is formed from the forward's o
before its own rounding (to 2^-16): that o has the weights' rounding, so do.o is off by at most
(2^-8 + E + 2^-16) sum |do| sum p |v|.  Sums over n keys or rows round n times at 2^-24.
"""

import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd.function import kda_attn, kda_qk_norm_rope
from oracle import around as A
from oracle import mixers as M
from test_gpu_around import DEV, Rand, dev, near, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(seed, B, Tq, Hq, Hk, D=128, past=0, lengths=None, pasts=None, rest=0, std=1.0):
    r, cq, ck = Rand(seed), None, None
    Tk = Tq + past
    if lengths is not None:
        B = 1
        cq = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32)
        keys = [n + p for n, p in zip(lengths, pasts or [past] * len(lengths))]
        ck = torch.tensor([0, *np.cumsum(keys)], dtype=torch.int32)
        Tq, Tk = int(cq[-1]) + rest, int(ck[-1]) + rest
    c = dict(q=r(B, Tq, Hq, D, dtype=BF, std=std), k=r(B, Tk, Hk, D, dtype=BF), v=r(B, Tk, Hk, D, dtype=BF), cq=cq, ck=ck,
             d_out=r(B, Tq, Hq, D, dtype=BF), d_lse=r(B, Tq, Hq), scale=D ** -0.5, N=B if cq is None else len(lengths),
             rest=rest)
    if rest:  # rows behind the last sequence hold nothing that may be used
        for n in ("q", "k", "v", "d_out", "d_lse"):
            c[n][:, c[n].shape[1] - rest:] = float("nan")
    return c


def seqs(c):
    tup = lambda t: None if t is None else t.tolist()  # noqa: E731
    q, k = c["q"], c["k"]
    return list(zip(A.bounds(q.shape[0], q.shape[1], tup(c["cq"])), A.bounds(k.shape[0], k.shape[1], tup(c["ck"]))))


def live(c, name):
    return A.f64(c[name].nan_to_num(0.0)).flatten(0, 1)


def expected(c, grad=True):
    """(values, tolerances) of out, lse, dq, dk, dv, from the formulas, head by head in fp64."""
    q, k, v, do, dl = (live(c, n) for n in ("q", "k", "v", "d_out", "d_lse"))
    Hq, Hk, D, sc = q.shape[1], k.shape[1], q.shape[2], c["scale"]
    val = dict(out=torch.zeros_like(q), lse=torch.full(q.shape[:2], -INF, dtype=torch.float64), dq=torch.zeros_like(q),
               dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    for (lo, hi), (a, z) in seqs(c):
        nq, nk = hi - lo, z - a
        if nq == 0 or nk == 0:
            continue
        sees = torch.arange(nk)[None] <= torch.arange(nq)[:, None] + (nk - nq)
        some = sees.any(1)
        for h in range(Hq):
            x, y, w, d, e = q[lo:hi, h], k[a:z, h * Hk // Hq], v[a:z, h * Hk // Hq], do[lo:hi, h], dl[lo:hi, h]
            s = torch.where(sees, sc * (x @ y.T), -INF)
            lse = torch.where(some, torch.logsumexp(torch.where(some[:, None], s, 0.0), -1), -INF)
            p = torch.where(some[:, None], torch.exp(s - lse.clamp(min=-1e300)[:, None]), 0.0)
            off = (130 * 2.0 ** -24 * sc * (x.abs() @ y.abs().T)).amax(-1, keepdim=True) * 2 + 2.0 ** -20  # E, twice
            o, size = p @ w, p @ w.abs()
            val["out"][lo:hi, h], val["lse"][lo:hi, h] = o, lse
            many = nk * 2.0 ** -24
            tol["out"][lo:hi, h] = (HALF + off + many) * size
            tol["lse"][lo:hi, h] = torch.where(some, off[:, 0] + many + 2.0 ** -22 * (1 + lse.abs()), 0.0)
            g = (d * o).sum(-1, keepdim=True) - e[:, None]
            dp = d @ w.T
            ds = p * (dp - g)
            dsz = p * (128 * 2.0 ** -24 * (d.abs() @ w.abs().T) + (HALF + off + many + 2.0 ** -15) * (d.abs() * size).sum(-1, keepdim=True)
                       + 2.0 ** -22 * e.abs()[:, None]) + (off + HALF + many) * ds.abs()
            val["dq"][lo:hi, h], tol["dq"][lo:hi, h] = sc * ds @ y, sc * dsz @ y.abs() + many * sc * ds.abs() @ y.abs()
            rows = nq * Hq // Hk * 2.0 ** -24
            val["dk"][a:z, h * Hk // Hq] += sc * ds.T @ x
            tol["dk"][a:z, h * Hk // Hq] += sc * (dsz + rows * ds.abs()).T @ x.abs()
            val["dv"][a:z, h * Hk // Hq] += p.T @ d
            tol["dv"][a:z, h * Hk // Hq] += (p * (off + HALF + rows)).T @ d.abs()
    for n in ("out", "dq", "dk", "dv"):
        tol[n] = tol[n] * (1 + HALF) + HALF * val[n].abs() + 1e-30
    return val, tol


def fwd(c, flags=0, keep=False):
    q, k, v = dev(c["q"]), dev(c["k"]), dev(c["v"])
    B, Tq, Hq, D = q.shape
    Tk, Hk = k.shape[1:3]
    out, lo = (torch.full(q.shape, 7.0, dtype=BF, device=DEV) for _ in range(2))
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    ws = torch.full((kda.kda_attn_workspace_size(B * Tq, B * Tk, Hq, Hk, D, c["N"]),), 255, dtype=torch.uint8, device=DEV)
    kda.kda_attn_fwd(q, k, v, c["scale"], out, lse, ws, lo if keep else None, dev(c["cq"]), dev(c["ck"]), flags)
    return (out, lse, lo) if keep else (out, lse)


def bwd(c, d_lse=True, flags=0):
    q, k, v = dev(c["q"]), dev(c["k"]), dev(c["v"])
    out, lse, lo = fwd(c, keep=True)
    dq, dk, dv = (torch.full(t.shape, 7.0, dtype=BF, device=DEV) for t in (q, k, v))
    ws = torch.full((kda.kda_attn_bwd_workspace_size(q.shape[0] * q.shape[1], k.shape[0] * k.shape[1], q.shape[2], k.shape[2],
                                                    q.shape[3], c["N"]),), 255, dtype=torch.uint8, device=DEV)
    kda.kda_attn_bwd(q, k, v, c["scale"], out, lo, lse, dev(c["d_out"]), dq, dk, dv, ws, dev(c["d_lse"]) if d_lse else None,
                     dev(c["cq"]), dev(c["ck"]), flags)
    return dq, dk, dv


def check(c, grad=True):
    val, tol = expected(c)
    got = dict(zip(("out", "lse"), fwd(c)))
    if grad:
        got |= dict(zip(("dq", "dk", "dv"), bwd(c)))
    for n, t in got.items():
        t = t.flatten(0, 1)
        M_ = t.shape[0] - c["rest"]
        want = val[n][:M_]
        if n == "lse":  # rows without keys exactly
            assert torch.equal(torch.isinf(t[:M_]).cpu(), torch.isinf(want))
            near(n, t[:M_].nan_to_num(neginf=0.0), want.nan_to_num(neginf=0.0), tol[n][:M_])
        else:
            near(n, t[:M_], want, tol[n][:M_])
        assert (t[M_:] == 7.0).all(), n  # rows of no sequence stay


WHOLE = {
    "one": (1, 1, 1, 1), "one_group": (2, 1, 8, 2, 64), "few": (1, 31, 2, 1), "tile": (1, 64, 2, 2), "tile_and_one": (1, 65, 3, 3, 64),
    "prompt": (1, 200, 2, 2), "odd_group": (2, 133, 10, 2, 64), "one_key_head": (1, 150, 7, 1), "many_tiles": (1, 700, 4, 2),
    "past": (1, 100, 4, 2, 128, 333), "past_odd": (2, 77, 6, 3, 64, 61), "token": (3, 1, 8, 2, 128, 1000),
    "token_far": (1, 1, 4, 1, 64, 5000), "tokens": (2, 5, 12, 4, 128, 1500), "big_group": (1, 3, 40, 1, 64, 700),
    "split_rows": (1, 700, 8, 1), "split_rows_two": (2, 1100, 6, 2, 64), "fewer_keys": (1, 90, 2, 1, 64, -30), "fewer_keys_tiles": (2, 300, 4, 2, 128, -70), "no_keys": (1, 20, 2, 1, 64, -20),
}
PACKED = {
    "ones": ([1, 1, 1], None, 0), "empties": ([0, 5, 0, 0, 64, 0], None, 3), "edges": ([63, 64, 65, 128, 1, 127, 129], None, 0),
    "all_empty": ([0, 0], None, 5), "pasts": ([3, 0, 40, 70, 1], [100, 7, 0, 33, 1], 40), "no_past_keys": ([30, 20], [-30, 4], 2),
    "fewer": ([130, 20, 9], [-70, -1, 2], 0), "long_among": ([1, 600, 2], [900, 0, 0], 9), "tokens": ([1] * 9, [1000, 0, 3, 700, 64, 63, 1, 2, 900], 0),
    "sixty_four": ([37 * i % 190 for i in range(64)], None, 7), "sixty_five": ([53 * i % 170 for i in range(65)], None, 0),
}


@pytest.mark.parametrize("name", WHOLE)
def test_batches(name):
    say("attention", name)
    check(case(300 + list(WHOLE).index(name), *WHOLE[name]))


@pytest.mark.parametrize("Hq,Hk,D", [(2, 2, 128), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("name", PACKED)
def test_packed(name, Hq, Hk, D):
    say("attention packed", name, Hq, Hk, D)
    lengths, pasts, rest = PACKED[name]
    check(case(330 + list(PACKED).index(name), 1, 0, Hq, Hk, D, lengths=lengths, pasts=pasts, rest=rest))


@pytest.mark.parametrize("std", [0.0, 20.0, 300.0])
def test_scores_from_equal_to_one_hot(std):
    """All scores zero; large ones, whose exponentials would overflow without the running maximum."""
    say("scores", std)
    check(case(350, 1, 150, 2, 1, std=std), grad=std < 100)


def test_a_maximum_that_keeps_rising():
    """Keys whose scores grow along the axis, so that every tile rescales what came before."""
    c = case(351, 1, 400, 2, 1, 64)
    c["q"] = torch.ones_like(c["q"])
    c["k"] = (torch.arange(400)[None, :, None, None] / 16.0 * torch.ones(1, 400, 1, 64)).to(BF)
    check(c, grad=False)


def test_one_row_sees_no_score_but_minus_infinity():
    """A key of infinities gives scores of minus infinity: such a row has no weight anywhere, as one without keys."""
    c = case(352, 1, 3, 1, 1, 64)
    c["q"], c["k"] = torch.ones_like(c["q"]), c["k"].clone()
    c["k"][0, 0] = -INF
    out, lse = fwd(c)
    assert (out[0, 0] == 0).all() and lse[0, 0, 0] == -INF and torch.isfinite(out.float()).all()
    val, tol = expected(dict(c, k=c["k"][:, 1:], v=c["v"][:, 1:], q=c["q"][:, 1:], d_out=c["d_out"][:, 1:], d_lse=c["d_lse"][:, 1:]))
    near("out", out[0, 1:], val["out"], tol["out"])


def test_nan_and_infinity_in_masked_places():
    """Keys of later tokens, keys and values of other sequences and rows of no sequence reach nobody."""
    c = case(353, 1, 0, 4, 2, lengths=[70, 64, 300], rest=50)
    clean = (*fwd(c), *bwd(c))
    b = dict(c, k=c["k"].clone(), v=c["v"].clone(), q=c["q"].clone())
    b["k"][0, 100], b["v"][0, 100, 0], b["q"][0, 100, 2:] = INF, float("nan"), float("nan")
    got = (*fwd(b), *bwd(b))
    for x, y in zip(got, clean):
        assert torch.equal(x[:, :70], y[:, :70]) and torch.equal(x[:, 134:434], y[:, 134:434])
    b = dict(c, k=c["k"].clone())
    b["k"][0, 130:134] = float("nan")  # the last keys of a sequence: earlier queries do not see them
    out, lse = fwd(b)
    assert torch.equal(out[:, 70:130], clean[0][:, 70:130]) and torch.equal(lse[:, 70:130], clean[1][:, 70:130])
    assert torch.isnan(out[:, 133].float()).all()


def test_strides_and_expanded_heads():
    r = Rand(360)
    B, T, Hq, Hk, D = 2, 150, 6, 2, 64
    wide = r(B, T, (Hq + 2 * Hk) * D + 8, dtype=BF).to(DEV).requires_grad_()
    def views(w):
        q, k, v, _ = w.split([Hq * D, Hk * D, Hk * D, 8], -1)
        return q.unflatten(-1, (Hq, D)), k.unflatten(-1, (Hk, D)), v.unflatten(-1, (Hk, D))
    d = r(B, T, Hq, D, dtype=BF).to(DEV)
    out, lse = kda_attn(*views(wide))
    (dw,) = torch.autograd.grad(out, wide, d)
    leaves = [t.detach().contiguous().requires_grad_() for t in views(wide)]
    o2, l2 = kda_attn(*leaves)
    g = torch.autograd.grad(o2, leaves, d)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert torch.equal(dw[..., :-8], torch.cat([t.flatten(2) for t in g], -1))
    # one key head expanded over several is the group's shared one
    one = leaves[1][:, :, :1].detach().requires_grad_()
    o3, _ = kda_attn(leaves[0], one.expand(B, T, 3, D), leaves[2][:, :, :1].expand(B, T, 3, D))
    o4, _ = kda_attn(leaves[0], one, leaves[2][:, :, :1])
    assert torch.equal(o3, o4)
    three = one.detach().expand(B, T, 3, D).contiguous().requires_grad_()
    o5, _ = kda_attn(leaves[0], three, leaves[2][:, :, :1].expand(B, T, 3, D))
    (g3,), (g4,), (parts,) = torch.autograd.grad(o3, one, d), torch.autograd.grad(o4, one, d), torch.autograd.grad(o5, three, d)
    # each head's part is rounded to bf16, and the sum of three twice in autograd's, once in the kernel's
    parts = parts.double().cpu()
    want, size = parts.sum(2, keepdim=True), parts.abs().sum(2, keepdim=True)
    near("dk", g3, want, 3 * HALF * size)
    near("dk", g4, want, 3 * HALF * size)


def test_a_prompt_in_pieces_is_the_whole_prompt():
    """Each piece of queries behind its past, down to single tokens, gives the whole prompt's rows."""
    c = case(361, 1, 300, 4, 2)
    out, lse = fwd(c)
    val, tol = expected(c)
    for lo, hi in [(0, 100), (100, 260), (260, 299), (299, 300)]:
        p = dict(c, q=c["q"][:, lo:hi], k=c["k"][:, :hi], v=c["v"][:, :hi])
        o, s = fwd(p)
        near("out", o[0], val["out"][lo:hi], tol["out"][lo:hi])
        near("lse", s[0], val["lse"][lo:hi], tol["lse"][lo:hi])


def test_results_of_split_keys_can_be_joined_by_their_log_sums():
    """lse is what a caller needs to join attention over two parts of the keys, with its gradient."""
    c = case(362, 2, 1, 4, 2, 64, past=200)
    q, k, v = (dev(c[n]) for n in ("q", "k", "v"))
    q = q.requires_grad_()
    (o1, l1), (o2, l2) = kda_attn(q, k[:, :90].contiguous(), v[:, :90].contiguous()), \
        kda_attn(q, k[:, 90:].contiguous(), v[:, 90:].contiguous())
    w = torch.softmax(torch.stack([l1, l2]), 0)[..., None]
    joined = w[0] * o1.float() + w[1] * o2.float()
    d = dev(c["d_out"])
    (g,) = torch.autograd.grad(joined, q, d.float())
    c["d_lse"].zero_()
    val, tol = expected(c)
    near("joined", joined.flatten(0, 1), val["out"], 3 * tol["out"] + 2.0 ** -8 * 2)
    near("dq", g.flatten(0, 1), val["dq"], 4 * tol["dq"] + 2.0 ** -7 * val["dq"].abs().max())


def test_gradients_are_differences_of_the_library():
    """Through lse, the fp32 result: along a direction in q and in k, steps that bf16 holds exactly."""
    c = case(363, 1, 60, 4, 2, 64)
    r = Rand(364)
    q, k = (torch.round(c[n].float() * 8) / 8 for n in ("q", "k"))
    u, w = (torch.sign(r(*t.shape)) / 64 for t in (q, k))
    c["d_out"].zero_()
    loss = lambda q, k: (fwd(dict(c, q=q.to(BF), k=k.to(BF)))[1].double().cpu() * c["d_lse"].double()).sum()  # noqa: E731
    q, k = q.clamp(-1.75, 1.75), k.clamp(-1.75, 1.75)
    assert all(torch.equal((t + s * x).to(BF).float(), t + s * x) for t, x in ((q, u), (k, w)) for s in (1, -1))
    dq, dk, _ = bwd(dict(c, q=q.to(BF), k=k.to(BF)))
    val, tol = expected(dict(c, q=q.to(BF), k=k.to(BF)))
    for g, x, n, args in ((dq, u, "dq", lambda s: (q + s * u, k)), (dk, w, "dk", lambda s: (q, k + s * w))):
        diff = (loss(*args(1)) - loss(*args(-1))) / 2
        got = (g.double().cpu() * x).sum()
        # a row's lse moves by a score change of at most a = 64 (1/64) 1.75/8; third derivative below 2 a^3
        third = 60 * 4 * 3 * (64 / 64 * 1.75 / 8) ** 3 / 3
        assert abs(diff - got) <= (tol[n].reshape(x.shape) * x.abs()).sum() + third


def test_only_one_of_the_results_is_used():
    c = case(365, 1, 90, 4, 2, 64)
    leaves = [dev(c[n]).requires_grad_() for n in ("q", "k", "v")]
    val, tol = expected(dict(c, d_lse=torch.zeros_like(c["d_lse"])))
    for n, g in zip(("dq", "dk", "dv"), torch.autograd.grad(kda_attn(*leaves)[0], leaves, dev(c["d_out"]))):
        near(n, g.flatten(0, 1), val[n], tol[n])
    val, tol = expected(dict(c, d_out=torch.zeros_like(c["d_out"])))
    g = torch.autograd.grad(kda_attn(*leaves)[1], leaves, dev(c["d_lse"]))
    for n, x in zip(("dq", "dk"), g):
        near(n, x.flatten(0, 1), val[n], tol[n])
    assert (g[2] == 0).all()


def test_rows_behind_the_last_sequence():
    c = case(366, 1, 0, 4, 2, 64, lengths=[30, 40], pasts=[5, 0], rest=100)
    leaves = [dev(c[n]).requires_grad_() for n in ("q", "k", "v")]
    out, lse = kda_attn(*leaves, cu_seqlens=dev(c["cq"]), cu_seqlens_k=dev(c["ck"]))
    g = torch.autograd.grad((out, lse), leaves, (dev(c["d_out"]), dev(c["d_lse"])))
    assert (out[:, 70:] == 0).all() and (lse[:, 70:] == -INF).all() and torch.isfinite(lse[:, :70]).all()
    assert (g[0][:, 70:] == 0).all() and (g[1][:, 75:] == 0).all() and (g[2][:, 75:] == 0).all()
    assert all(torch.isfinite(t.float()).all() for t in g)


def test_the_same_bits_every_time():
    c = case(367, 1, 0, 6, 2, lengths=[300, 1, 200], pasts=[0, 900, 50])
    assert all(torch.equal(x, y) for x, y in zip((*fwd(c), *bwd(c)), (*fwd(c), *bwd(c))))
    t = case(368, 2, 1, 8, 2, past=3000)
    assert all(torch.equal(x, y) for x, y in zip(fwd(t), fwd(t)))


def test_captured_and_replayed_among_eager_calls():
    c, t = case(369, 1, 0, 4, 2, 64, lengths=[200, 0, 90]), case(370, 2, 1, 8, 2, past=3000)
    leaves = [dev(c[n]).requires_grad_() for n in ("q", "k", "v")]
    token = [dev(t[n]) for n in ("q", "k", "v")]
    cu, cot = dev(c["cq"]), dev(c["d_out"])

    def step():
        out, lse = kda_attn(*leaves, cu_seqlens=cu)
        return (out.detach(), lse.detach(), *torch.autograd.grad(out, leaves, cot), *kda_attn(*token))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        with torch.no_grad():
            for x in (*leaves, *token):
                x.copy_(Rand(400 + i)(*x.shape, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        del want


def test_two_streams_with_their_own_workspaces():
    a, b = case(371, 4, 1, 8, 2, past=3000), case(372, 1, 1, 4, 1, past=4000)
    want = fwd(a), fwd(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        x = fwd(a)
    with torch.cuda.stream(s2):
        y = fwd(b)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*x, *y), (*want[0], *want[1])))


def test_no_queries_no_keys():
    q, k = torch.empty(2, 0, 4, 64, dtype=BF, device=DEV), torch.randn(2, 5, 2, 64, device=DEV).to(BF).requires_grad_()
    out, lse = kda_attn(q, k, k)
    assert out.shape == q.shape and lse.shape == (2, 0, 4)
    (g,) = torch.autograd.grad(out, k, torch.empty_like(out))
    assert (g == 0).all()
    q, k = k.detach().repeat(1, 1, 2, 1), torch.empty(2, 0, 2, 64, dtype=BF, device=DEV)
    out, lse = kda_attn(q, k, k)
    assert (out == 0).all() and (lse == -INF).all()


def test_behind_the_norm_and_rotation():
    """A full-attention layer's path: one projection's output, rows normed with weights and turned, attention."""
    r = Rand(373)
    B, T, Hq, Hk, D = 1, 130, 8, 2, 64
    wide = r(B, T, Hq + 2 * Hk, D, dtype=BF).to(DEV).requires_grad_()
    qw, kw = ((1 + r(D, std=0.2)).to(DEV).requires_grad_() for _ in range(2))
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV)[None], torch.full((D // 2,), 0.3, dtype=torch.float64, device=DEV)
    q, k = kda_qk_norm_rope(wide[:, :, :Hq], wide[:, :, Hq:Hq + Hk], pos, f, q_weight=qw, k_weight=kw, norm="rms")
    out, lse = kda_attn(q, k, wide[:, :, Hq + Hk:])
    d = r(*out.shape, dtype=BF)
    g = torch.autograd.grad(out, [wide, qw, kw], d.to(DEV))
    c = dict(q=q.detach().cpu(), k=k.detach().cpu(), v=wide[:, :, Hq + Hk:].detach().cpu(), cq=None, ck=None, d_out=d,
             d_lse=torch.zeros(B, T, Hq), scale=D ** -0.5, rest=0)
    val, tol = expected(c)
    near("out", out.flatten(0, 1), val["out"], tol["out"])
    near("dv", g[0][:, :, Hq + Hk:].flatten(0, 1), val["dv"], tol["dv"])
    assert all(torch.isfinite(t.float()).all() and t.float().abs().max() > 0 for t in g)
