"""The token mixers on two streams at once, each call with a workspace and outputs of its own, all of them there
before the first call is enqueued."""

import pytest
import torch

import chunked_gated_delta_amd as kda
import test_gpu_attn as at
import test_gpu_linear_attn as la
from test_gpu_around import DEV, dev, say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CALLS = 6  # on each stream


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def scratch(n):
    return torch.full((n,), 255, dtype=torch.uint8, device=DEV)


def like(*ts):
    return [torch.full_like(t, 7.0) for t in ts]


def attn(c, grad):
    """(the call for outputs of its own, made beforehand)"""
    q, k, v, cq, ck, do, dl = (dev(c[n]) for n in ("q", "k", "v", "cq", "ck", "d_out", "d_lse"))
    sizes = (q.shape[0] * q.shape[1], k.shape[0] * k.shape[1], q.shape[2], k.shape[2], q.shape[3], c["N"])
    need = (kda.kda_attn_workspace_size(*sizes), kda.kda_attn_bwd_workspace_size(*sizes))
    lse = torch.full(q.shape[:3], 7.0, device=DEV)

    def make():
        out, lo, s, dq, dk, dv, ws, wb = *like(q, q, lse, q, k, v), *map(scratch, need)

        def call():
            kda.kda_attn_fwd(q, k, v, c["scale"], out, s, ws, lo, cq, ck)
            if grad:
                kda.kda_attn_bwd(q, k, v, c["scale"], out, lo, s, do, dq, dk, dv, wb, dl, cq, ck)
        return call, [out, lo, s, dq, dk, dv]
    return make


def linear(c):
    q, k, v, g, init, cu, do, df = (dev(c[n]) for n in ("q", "k", "v", "g", "init", "cu", "d_out", "d_fin"))
    B, T, H, K = q.shape
    V, N = v.shape[3], c["N"]
    need = (kda.kda_la_workspace_size(B * T, H, K, V), kda.kda_la_bwd_workspace_size(B * T, H, K, V, N))

    def make():
        out, fin, dq, dk, dv, dg, di, ws, wb = *like(v, df, q, k, v, g, df), *map(scratch, need)

        def call():
            kda.kda_la_fwd(q, k, v, g, c["scale"], out, ws, init, fin, cu)
            kda.kda_la_bwd(q, k, v, g, c["scale"], do, dq, dk, dv, wb, dg, init, df, di, cu)
        return call, [out, fin, dq, dk, dv, dg, di]
    return make


PAIRS = {
    "tokens": lambda: (attn(at.case(560, 16, 1, 8, 2, past=3000), False), attn(at.case(561, 1, 1, 4, 1, past=60000), False)),
    "attention": lambda: (attn(at.case(562, 1, 700, 8, 1), True), attn(at.case(563, 1, 0, 6, 2, lengths=[300, 1, 900], pasts=[0, 900, 50]), True)),
    "linear": lambda: (linear(la.case(564, 1, 4000, 4)), linear(la.case(565, 1, 0, 3, lengths=[2900, 0, 700, 3]))),
    "both": lambda: (linear(la.case(566, 2, 2000, 3)), attn(at.case(567, 2, 1, 8, 2, past=20000), True)),
}


@pytest.mark.parametrize("name", PAIRS)
def test_calls_on_two_streams_with_their_own_workspaces(name):
    say("two streams", name)
    pair = PAIRS[name]()
    alone = []
    for make in pair:
        call, outs = make()
        call()
        torch.cuda.synchronize()
        alone.append(outs)
    ready = [[make() for _ in range(CALLS)] for make in pair]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(CALLS):
        for s, calls in zip(streams, ready):
            with torch.cuda.stream(s):
                calls[i][0]()
    torch.cuda.synchronize()
    for want, calls in zip(alone, ready):
        for _, got in calls:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
