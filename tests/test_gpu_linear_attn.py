"""Linear attention with a decay for each head on the GPU against its fp64 oracle (oracle/mixers.py).

Tolerances, with A(x) the same sum over the absolute values of its terms:

* bf16 results: half a step of the value (2^-8), plus 2^-15 A for the pair weights and entering states
  that are split in two bf16 parts (2^-8 2^-8 each), plus the
  roundings of fp32 sums, 2^-24 A each: up to 128 channels, 64 tokens, and, in a state, 64 tokens and
  two products for each of the steps that it was carried over.
* states and the decay's gradient, fp32 results: three parts (2^-24), and the same sums.
"""

import numpy as np
import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd.function import kda_linear_attn
from oracle import around as A
from oracle import mixers as M
from test_gpu_around import DEV, Rand, dev, near, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def case(seed, B, T, H, K=128, V=128, lengths=None, rest=0, init=True, g=None):
    r, cu = Rand(seed), None
    if lengths is not None:
        cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32)
        B, T = 1, int(cu[-1]) + rest
    N = B if cu is None else len(lengths)
    c = dict(q=r(B, T, H, K, dtype=BF), k=r(B, T, H, K, dtype=BF), v=r(B, T, H, V, dtype=BF),
             g=-torch.exp(r(H, std=2.0) - 3.0) if g is None else torch.tensor(g, dtype=torch.float32),
             init=r(N, H, K, V) if init else None, cu=cu, d_out=r(B, T, H, V, dtype=BF), d_fin=r(N, H, K, V),
             scale=K ** -0.5, N=N)
    if rest:  # rows behind the last sequence hold nothing that may be used
        for n in ("q", "k", "v", "d_out"):
            c[n][:, T - rest:] = float("nan")
    return c


def oracle(c, grad=True, absolute=False):
    cu = None if c["cu"] is None else c["cu"].tolist()
    f = lambda q, k, v, g, i: M.linear_attn(q, k, v, g, i, cu, c["scale"])  # noqa: E731
    size = (lambda t: None if t is None else t.abs()) if absolute else (lambda t: t)
    live = [size(None if c[n] is None else c[n].nan_to_num(0.0)) for n in ("q", "k", "v")]
    leaves = [*live, c["g"], size(c["init"])]
    if not grad:
        return f(*(A.f64(t) for t in leaves)), None
    return A.grads(f, leaves, [size(c["d_out"].nan_to_num(0.0)), size(c["d_fin"])])


def carried(c):
    T = c["q"].shape[1]
    longest = T if c["cu"] is None else int((c["cu"][1:] - c["cu"][:-1]).max())
    return (longest // 64 + 3) * 66 * 2.0 ** -24


def tolerances(c, absolute):
    (out, fin), g = absolute
    steps = carried(c) + 256 * 2.0 ** -24
    some = 2.0 ** -15 + steps
    return [some * out, steps * fin], [*(some * t for t in g[:3]), (2.0 ** -23 + steps) * g[3],
                                       None if c["init"] is None else steps * g[4]]


def fwd(c, out=None, flags=0):
    q, k, v = dev(c["q"]), dev(c["k"]), dev(c["v"])
    B, T, H, K = q.shape
    V = v.shape[3]
    out = torch.full((B, T, H, V), 7.0, dtype=BF, device=DEV) if out is None else out
    fin = torch.full((c["N"], H, K, V), float("nan"), device=DEV)
    ws = torch.full((kda.kda_la_workspace_size(B * T, H, K, V),), 255, dtype=torch.uint8, device=DEV)
    kda.kda_la_fwd(q, k, v, dev(c["g"]), c["scale"], out, ws, dev(c["init"]), fin, dev(c["cu"]), flags)
    return out, fin


def bwd(c, dg=True, final=True, flags=0):
    q, k, v = dev(c["q"]), dev(c["k"]), dev(c["v"])
    B, T, H, K = q.shape
    V = v.shape[3]
    dq, dk, dv = (torch.full(t.shape, 7.0, dtype=BF, device=DEV) for t in (q, k, v))
    g = torch.full((H,), float("nan"), device=DEV) if dg else None
    di = None if c["init"] is None else torch.full((c["N"], H, K, V), float("nan"), device=DEV)
    ws = torch.full((kda.kda_la_bwd_workspace_size(B * T, H, K, V, c["N"]),), 255, dtype=torch.uint8, device=DEV)
    kda.kda_la_bwd(q, k, v, dev(c["g"]), c["scale"], dev(c["d_out"]), dq, dk, dv, ws, g, dev(c["init"]),
                   dev(c["d_fin"]) if final else None, di, dev(c["cu"]), flags)
    return dq, dk, dv, g, di


CASES = {
    "one": (1, 1, 1, 128, 128), "two_short": (2, 17, 3, 128, 64), "step": (1, 64, 2, 64, 64), "step_and_one": (1, 65, 2, 64, 128),
    "prompt": (1, 200, 2, 128, 128), "segments": (2, 1300, 1, 128, 128), "segments_odd": (1, 2111, 2, 64, 128),
    "segments_wide": (1, 1025, 3, 128, 64), "whole": (1, 150, 90, 64, 64),
}
PACKED = {
    "one_each": [1, 1, 1], "empty": [0, 5, 0, 0, 64, 0], "edges": [63, 64, 65, 128, 1], "all_empty": [0, 0],
    "across": [700, 3, 0, 900, 511, 1, 512], "long_among": [1, 1999, 2],
}


def all_cases():
    for n, (i, s) in zip(CASES, enumerate(CASES.values())):
        yield n, lambda i=i, s=s: case(100 + i, *s, init=i % 2 == 0)
    for i, (n, lengths) in enumerate(PACKED.items()):
        yield "packed_" + n, lambda i=i, x=lengths: case(120 + i, 1, 0, 2, (64, 128)[i % 2], (128, 128, 64)[i % 3], lengths=x,
                                                         rest=i % 3 * 40, init=i % 4 != 3)


ALL = dict(all_cases())


@pytest.mark.parametrize("name", ALL)
def test_forward_and_gradients(name):
    say("linear attention", name)
    c = ALL[name]()
    rest = c["q"].shape[1] - (c["q"].shape[1] if c["cu"] is None else int(c["cu"][-1]))
    (out, fin), grads = oracle(c)
    t_out, t_grad = tolerances(c, oracle(c, absolute=True))
    got = fwd(c)
    near("final", got[1], fin, t_out[1])
    M_ = got[0].shape[0] * got[0].shape[1]
    live = slice(0, M_ - rest)
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    near("out", flat(got[0])[live], out[live], HALF * out[live].abs() + t_out[0][live])
    assert (flat(got[0])[M_ - rest:] == 7.0).all()  # rows of no sequence stay
    g = bwd(c)
    for n, x, want, tol in zip(("dq", "dk", "dv"), g, grads, t_grad):
        want, tol = flat(want), flat(tol)
        near(n, flat(x)[live], want[live], HALF * want[live].abs() + tol[live])
        assert (flat(x)[M_ - rest:] == 7.0).all()
    near("d_log_decay", g[3], grads[3], t_grad[3] + 1e-30)
    if c["init"] is not None:
        near("d_initial_state", g[4], grads[4], t_grad[4])


def test_states_and_the_decays_gradient_are_fp32_results():
    """Two bf16 parts in place of three would leave 4e-6 of the norm; fp32 sums leave about 1e-7, and the
    gradient's sums over all tokens, of either sign, some times that."""
    c = case(150, 1, 1500, 8, g=[-2.0 ** -i for i in range(8)])
    (_, fin), grads = oracle(c)
    got, g = fwd(c)[1], bwd(c)
    rel = lambda x, y: ((x.double().cpu() - y).norm() / y.norm()).item()  # noqa: E731
    assert rel(got, fin) < 2.0 ** -20 and rel(g[4], grads[4]) < 2.0 ** -20
    size = oracle(c, absolute=True)[1][3]
    assert ((g[3].double().cpu() - grads[3]).abs() < 2.0 ** -20 * size).all()


@pytest.mark.parametrize("g", [0.0, -1e-30, -2.0 ** -12, -5.0, -60.0, -200.0])
def test_decays_from_none_to_all(g):
    say("decay", g)
    c = case(160, 1, 700, 2, 64, 64, g=[g, -0.1])
    (out, fin), grads = oracle(c)
    t_out, t_grad = tolerances(c, oracle(c, absolute=True))
    got, d = fwd(c), bwd(c)
    near("out", got[0].flatten(0, 1), out, HALF * out.abs() + t_out[0])
    near("final", got[1], fin, t_out[1] + 1e-37)
    for n, x, want, tol in zip(("dq", "dk", "dv", "dg", "di"), d, grads, t_grad):
        near(n, x, want, (HALF * want.abs() if n[1] in "qkv" else 0) + tol + 1e-37)


def test_a_decay_of_minus_infinity_keeps_nothing():
    c = case(161, 2, 130, 2, g=[-float("inf"), -float("inf")])
    got, d = fwd(c), bwd(c)
    (out, fin), _ = oracle(c, grad=False)
    near("out", got[0].flatten(0, 1), out, HALF * out.abs() + 2.0 ** -14 * out.abs().max())
    near("final", got[1], fin, 2.0 ** -22 * fin.abs())
    assert (d[3] == 0).all() and (d[4] == 0).all() and all(torch.isfinite(t.float()).all() for t in d[:3])


def test_strides_and_shared_heads():
    """Slices of one projection's output; one head's keys for all of them, whose gradient is a sum."""
    r = Rand(170)
    B, T, H, K, V = 2, 150, 3, 64, 128
    wide = r(B, T, H * (K + V) + 64 + 8, dtype=BF).to(DEV)
    q, v, k = wide.split([H * K, H * V, 64 + 8], -1)
    q, v, k = q.unflatten(-1, (H, K)), v.unflatten(-1, (H, V)), k[..., :K].unsqueeze(2).expand(B, T, H, K)
    g = -torch.rand(H, device=DEV)
    want = kda_linear_attn(q.contiguous(), k.contiguous(), v.contiguous(), g)
    got = kda_linear_attn(q, k, v, g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide.requires_grad_()
    q, v, k = wide.split([H * K, H * V, 64 + 8], -1)
    one = k[..., :K].unsqueeze(2)
    d = r(B, T, H, V, dtype=BF).to(DEV)
    (dw,) = torch.autograd.grad(kda_linear_attn(q.unflatten(-1, (H, K)), one.expand(B, T, H, K), v.unflatten(-1, (H, V)), g)[0],
                                wide, d)
    leaves = [t.detach().contiguous().requires_grad_() for t in
              (q.unflatten(-1, (H, K)), one.expand(B, T, H, K), v.unflatten(-1, (H, V)))]
    dq, dk, dv = torch.autograd.grad(kda_linear_attn(*leaves, g)[0], leaves, d)
    assert torch.equal(dw[..., :H * K], dq.flatten(2)) and torch.equal(dw[..., H * K:H * (K + V)], dv.flatten(2))
    near("shared", dw[..., H * (K + V):][..., :K], dk.double().sum(2).cpu(), 2 * HALF * dk.double().abs().sum(2).cpu())


def test_a_nan_stays_in_its_sequence_and_head():
    c = case(171, 1, 0, 3, lengths=[70, 64, 300])
    clean, dclean = fwd(c), bwd(c)
    for n in ("q", "k", "v", "d_out"):
        b = dict(c)
        b[n] = c[n].clone()
        b[n][0, 100, 1] = float("inf") if n == "k" else float("nan")
        got, d = fwd(b), bwd(b)
        for x, y in ((got[0], clean[0]), *zip(d[:3], dclean[:3])):
            assert torch.equal(x[:, :70], y[:, :70]) and torch.equal(x[:, 134:], y[:, 134:])
            assert torch.equal(x[:, :, [0, 2]], y[:, :, [0, 2]])
        assert torch.equal(got[1][[0, 2]], clean[1][[0, 2]]) and torch.equal(d[3][[0, 2]], dclean[3][[0, 2]])


def test_split_run_equals_whole_run():
    """The final state of the first part is the initial state of the second."""
    c = case(172, 1, 1100, 2, g=[-0.01, -0.3])
    out, fin = fwd(c)
    a = dict(c, **{n: c[n][:, :401] for n in ("q", "k", "v")})
    first = fwd(a)
    b = dict(c, init=first[1].cpu(), **{n: c[n][:, 401:] for n in ("q", "k", "v")})
    second = fwd(b)
    size = oracle(c, grad=False, absolute=True)[0]
    near("out", torch.cat([first[0], second[0]], 1).flatten(0, 1), out.double().cpu().flatten(0, 1),
         2 * HALF * out.double().cpu().abs().flatten(0, 1) + (2.0 ** -14 + 2 * carried(c)) * size[0])
    near("final", second[1], fin.double().cpu(), 2 * carried(c) * size[1])


@pytest.mark.parametrize("B,T,H,K,V", [(1, 1, 1, 128, 128), (5, 1, 3, 64, 128), (2, 3, 7, 128, 64), (3, 7, 2, 64, 64), (2, 0, 2, 64, 64)])
def test_step(B, T, H, K, V):
    say("step", B, T, H, K, V)
    c = case(180 + B, B, T, H, K, V)
    (out, fin), _ = oracle(c, grad=False)
    (a_out, a_fin), _ = oracle(c, grad=False, absolute=True)
    q, k, v, g, state = (dev(c[n]) for n in ("q", "k", "v", "g", "init"))
    o = torch.empty(B, T, H, V, dtype=BF, device=DEV)
    f = torch.full_like(state, float("nan"))
    kda.kda_la_step(q, k, v, g, c["scale"], o, initial_state=state, final_state=f)
    # a token's state: its decay (2 roundings), a product and a sum; outputs sum 128 channels more
    near("out", o.flatten(0, 1), out, HALF * out.abs() + (4 * T + 140) * 2.0 ** -24 * a_out)
    near("final", f, fin, (4 * T + 4) * 2.0 ** -24 * a_fin)
    kda.kda_la_step(q, k, v, g, c["scale"], o, initial_state=state, final_state=state)  # in place
    assert torch.equal(state, f)
    o2 = torch.empty_like(o)
    kda.kda_la_step(q, k, v, g, c["scale"], o2)  # from zeros, state not wanted
    zero = dict(c, init=None)
    want, size = oracle(zero, grad=False)[0][0], oracle(zero, grad=False, absolute=True)[0][0]
    near("out", o2.flatten(0, 1), want, HALF * want.abs() + (4 * T + 140) * 2.0 ** -24 * size)


def test_prompt_then_tokens():
    """A prompt's state goes on token by token as one longer prompt would."""
    c = case(190, 1, 140, 2, init=False)
    out, fin = fwd(c)
    head = dict(c, **{n: c[n][:, :137] for n in ("q", "k", "v")})
    o, state = fwd(head)
    size = oracle(c, grad=False, absolute=True)[0]
    for t in range(137, 140):
        x = [dev(c[n][:, t:t + 1].contiguous()) for n in ("q", "k", "v")]
        step = torch.empty_like(x[2])
        kda.kda_la_step(*x, dev(c["g"]), c["scale"], step, initial_state=state, final_state=state)
        near("token", step[:, 0], out[:, t].double().cpu(), 2 * HALF * out[:, t].double().cpu().abs() + 2.0 ** -14 * size[0][t])
    near("state", state, fin.double().cpu(), 2 * carried(c) * size[1])


def test_the_same_bits_every_time():
    c = case(191, 1, 0, 2, lengths=[700, 900, 5])
    a, b = (fwd(c), bwd(c)), (fwd(c), bwd(c))
    assert all(torch.equal(x, y) for x, y in zip((*a[0], *a[1]), (*b[0], *b[1])))


@pytest.mark.parametrize("which", ["initial_state", "log_decay", "fewest"])
def test_only_the_gradients_that_are_asked_for(which):
    c = case(192, 1, 130, 2, 64, 64)
    t = {n: dev(c[n]) for n in ("q", "k", "v")} | dict(log_decay=dev(c["g"]), initial_state=dev(c["init"]))
    every = {n: x.detach().requires_grad_() for n, x in t.items()}
    call = lambda d: kda_linear_attn(d["q"], d["k"], d["v"], d["log_decay"], initial_state=d["initial_state"])  # noqa: E731
    cot = (dev(c["d_out"]), dev(c["d_fin"]))
    want = dict(zip(every, torch.autograd.grad(call(every), list(every.values()), cot)))
    n = "v" if which == "fewest" else which
    some = dict(t) | {n: t[n].detach().requires_grad_()}
    (got,) = torch.autograd.grad(call(some), [some[n]], cot)
    assert torch.equal(got, want[n])
    some = dict(t) | {n: t[n].detach().requires_grad_()}  # from one of the outputs alone
    (got,) = torch.autograd.grad(call(some)[1], [some[n]], cot[1])
    _, g = A.grads(lambda q, k, v, g, i: M.linear_attn(q, k, v, g, i, None, c["scale"]),
                   [c["q"], c["k"], c["v"], c["g"], c["init"]], [None, c["d_fin"]])
    want = g[["q", "k", "v", "log_decay", "initial_state"].index(n)]
    near(n, got, want, HALF * want.abs() + 2.0 ** -12 * want.abs().max())


def test_gradients_are_differences_of_the_library():
    """In the two fp32 inputs, through the fp32 output: the final state is linear in the initial one,
    and its second derivative in the decay bounds the difference quotient's error."""
    c = case(193, 1, 300, 2, 64, 64, g=[-0.02, -0.4])
    c["d_out"].zero_()
    d = bwd(c)
    loss = lambda x: (fwd(x)[1].double().cpu() * c["d_fin"].double()).sum()  # noqa: E731
    size = (oracle(c, absolute=True)[0][1] * c["d_fin"].double().abs()).sum()
    move = Rand(194)(*c["init"].shape)
    diff = loss(dict(c, init=c["init"] + move)) - loss(c)
    assert abs(diff - (d[4].double().cpu() * move.double()).sum()) <= 2 * carried(c) * 2 * size
    h = 2.0 ** -10
    for i in range(2):
        up, down = (dict(c, g=c["g"] + s * h * torch.eye(2)[i]) for s in (1, -1))
        diff = (loss(up) - loss(down)) / ((up["g"] - down["g"])[i].double())
        # third derivative: at most 300^3 tokens^3 of the size where the memory is long, divided by 6
        reach = min(300.0, 3.0 / abs(c["g"][i].item())) ** 3
        assert abs(diff - d[3][i].double().cpu()) <= (2 * carried(c) / h + h * h * reach / 6) * size


def test_captured_and_replayed_among_eager_calls():
    c = case(195, 1, 0, 2, lengths=[700, 0, 450])
    leaves = [dev(c[n]).requires_grad_() for n in ("q", "k", "v", "g", "init")]
    cu, cot = dev(c["cu"]), (dev(c["d_out"]), dev(c["d_fin"]))

    def step():
        outs = kda_linear_attn(*leaves[:4], initial_state=leaves[4], cu_seqlens=cu)
        return (*(o.detach() for o in outs), *torch.autograd.grad(outs, leaves, cot))

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
            for x in leaves[:3]:
                x.copy_(Rand(200 + i)(*x.shape, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        del want


def test_two_streams_with_their_own_workspaces():
    a, b = case(196, 1, 1500, 2), case(197, 1, 900, 3)
    want = fwd(a), fwd(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        x = fwd(a)
    with torch.cuda.stream(s2):
        y = fwd(b)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*x, *y), (*want[0], *want[1])))


def test_rows_behind_the_last_sequence_come_back_as_zeros():
    c = case(198, 1, 0, 2, 64, 128, lengths=[30, 40], rest=100)
    leaves = [dev(c[n]).requires_grad_() for n in ("q", "k", "v")]
    out, _ = kda_linear_attn(*leaves, dev(c["g"]), cu_seqlens=dev(c["cu"]))
    g = torch.autograd.grad(out, leaves, dev(c["d_out"]))
    assert all((t[:, 70:] == 0).all() and torch.isfinite(t.float()).all() for t in (out, *g))


def test_no_tokens_and_no_gradient():
    q = torch.empty(2, 0, 3, 64, dtype=BF, device=DEV)
    init = torch.randn(2, 3, 64, 64, device=DEV)
    out, fin = kda_linear_attn(q, q, q, torch.zeros(3, device=DEV), initial_state=init)
    assert out.shape == q.shape and torch.equal(fin, init) and fin.grad_fn is None
    leaf = init.clone().requires_grad_()
    g = torch.zeros(3, device=DEV, requires_grad=True)
    fin = kda_linear_attn(q, q, q, g, initial_state=leaf)[1]
    d = torch.autograd.grad(fin, [leaf, g], init)
    assert torch.equal(d[0], init) and (d[1] == 0).all()
