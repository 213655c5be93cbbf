"""Linear attention where nothing is kept from one token to the next, against the closed form: with a decay of
exp(-inf) = 0 the state is the last token's k v^T alone, so that

    out_t = scale (q_t.k_t) v_t,   dq_t = scale (v_t.do_t) k_t,   dk_t = scale (v_t.do_t) q_t,   dv_t = scale (q_t.k_t) do_t,

and the last token of a sequence has dS v_t in dk_t and dS^T k_t in dv_t as well, for the gradient dS of the final
state.  The decay's and the initial state's gradients are zero (but for a sequence without tokens, whose initial
state is its final one).  Tolerances as in test_gpu_linear_attn.py, A being the sums over absolute values.
"""

import pytest
import torch

from oracle import around as A
from test_gpu_around import near, say
from test_gpu_linear_attn import HALF, bwd, carried, case, fwd

pytestmark = pytest.mark.gpu
NONE = -float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def closed(c, size=lambda t: t):
    q, k, v, do, df, init = (size(A.f64(c[n].nan_to_num(0.0))) for n in ("q", "k", "v", "d_out", "d_fin", "init"))
    B, T = q.shape[:2]
    q, k, v, do = (t.flatten(0, 1) for t in (q, k, v, do))
    qk, vd, sc = (q * k).sum(-1, keepdim=True), (v * do).sum(-1, keepdim=True), c["scale"]
    out, dq, dk, dv = sc * qk * v, sc * vd * k, sc * vd * q, sc * qk * do
    fin, di = init.clone(), df.clone()
    for n, (lo, hi) in enumerate(A.bounds(B, T, None if c["cu"] is None else c["cu"].tolist())):
        if hi > lo:
            x, y, z = df[n], k[hi - 1], v[hi - 1]
            fin[n] = y[:, :, None] * z[:, None]
            dk[hi - 1] += (x * z[:, None]).sum(-1)
            dv[hi - 1] += (x * y[:, :, None]).sum(-2)
            di[n] = 0
    return out, fin, dq, dk, dv, di


@pytest.mark.parametrize("name,args,kw", [
    ("two", (2, 130, 2), {}), ("token", (3, 1, 2, 64, 128), {}), ("segments", (1, 2111, 2, 64, 64), {}),
    ("segments_wide", (1, 1300, 1, 128, 64), {}), ("packed", (1, 0, 2), dict(lengths=[0, 700, 1, 65, 0, 512, 64], rest=9))])
def test_a_decay_of_minus_infinity_against_the_closed_form(name, args, kw):
    say("nothing is kept", name)
    c = case(570, *args, **kw)
    c["g"] = torch.full_like(c["g"], NONE)
    want, size = closed(c), closed(c, torch.abs)
    some = 2.0 ** -15 + carried(c) + 256 * 2.0 ** -24
    got = (*fwd(c), *(d := bwd(c))[:3], d[4])
    live = c["q"].shape[0] * c["q"].shape[1] - kw.get("rest", 0)
    for n, g, w, s in zip(("out", "final", "dq", "dk", "dv", "d_initial_state"), got, want, size):
        if n in ("final", "d_initial_state"):
            near(n, g, w, (carried(c) + 256 * 2.0 ** -24) * s)
        else:
            near(n, g.flatten(0, 1)[:live], w[:live], HALF * w[:live].abs() + some * s[:live])
    assert (d[3] == 0).all()


def test_heads_that_keep_nothing_beside_heads_that_do():
    """The gradients of a head with a decay are the same bits beside one without any."""
    c = case(571, 1, 500, 2, 64, 64, g=[-0.05, -0.05])
    both, one = (*fwd(c), *bwd(c)), dict(c, g=torch.tensor([-0.05, NONE]))
    got = (*fwd(one), *bwd(one))
    for x, y in zip(got, both):
        assert torch.equal(x[0] if x.dim() == 1 else x[:, 0] if x.dtype == torch.float32 else x[:, :, 0],
                           y[0] if y.dim() == 1 else y[:, 0] if y.dtype == torch.float32 else y[:, :, 0])
