"""Sizes at the limits of what one call of a token mixer takes (CPU only: every call here is rejected before any
device work, so its pointers are never dereferenced)."""

import pytest
import torch

import chunked_gated_delta_amd as kda
from test_boundary_mixers import INVALID, P, Meta, at_bwd, at_fwd, la_bwd, la_fwd, la_step

M = 1 << 20


@pytest.mark.parametrize("call,sizes", [
    # workgroups of 256 threads, one for a head of a sequence and 64 of its output's channels
    (la_fwd, dict(B=M, N=M, H=16, T=1)), (la_fwd, dict(B=M, N=M, H=16, T=1, K=128)), (la_fwd, dict(B=M, N=M, H=8, T=1, V=128)),
    (la_fwd, dict(B=M, N=M, H=16, T=0)),
    # dq would fit, dv and dk in one launch, or either in its own, would not
    (la_bwd, dict(B=M, N=M, H=8, T=1)), (la_bwd, dict(B=M, N=M, H=4, T=1, K=128, V=128)), (la_bwd, dict(B=M, N=M, H=8, T=1, V=128)),
    (la_bwd, dict(B=M, N=M, H=8, T=1, K=128)), (la_bwd, dict(B=M, N=M, H=8, T=1, dg=P[12], dfin=P[13], di=P[14])),
    (la_step, dict(B=M, H=16, T=1)), (la_step, dict(B=M, H=16, T=0)), (la_step, dict(B=16, H=M, T=1)),
    # tiles of one wave, and of four
    (at_fwd, dict(B=M, N=M, Tq=1, Tk=1, Hq=64, Hk=64)), (at_fwd, dict(N=M, Tq=M, Tk=M, Hq=64, Hk=64, cq=P[17], ck=P[18])),
    (at_fwd, dict(B=1 << 17, N=1 << 17, Tq=129, Tk=300, Hq=64, Hk=64)),
    # 512 threads a tile of keys, with gradients; few keys, but many tiles of rows; rows and heads of the sums do.o
    (at_bwd, dict(N=M, Tq=M, Tk=M, Hq=8, Hk=8, cq=P[17], ck=P[18])), (at_bwd, dict(B=M, N=M, Tq=1, Tk=1, Hq=8, Hk=8)),
    (at_bwd, dict(B=1 << 18, N=1 << 18, Tq=1 << 13, Tk=1, Hq=1, Hk=1)), (at_bwd, dict(B=1 << 17, N=1 << 17, Tq=129, Tk=0, Hq=1 << 15, Hk=1)),
])
def test_more_threads_than_a_launch_has_are_refused(call, sizes):
    """Before the first of a call's launches: gradients are written by all of them or by none."""
    assert call(**sizes) == INVALID


def test_the_first_keys_of_a_longer_cache(monkeypatch):
    """Of one sequence they are taken as they lie; of several there is no stride between sequences, and they
    are refused rather than read from the wrong rows."""
    monkeypatch.setattr(kda, "_Call", Meta)
    bf = torch.bfloat16
    q, cache = torch.zeros(3, 1, 4, 64, dtype=bf), torch.zeros(3, 10, 2, 64, dtype=bf)
    for k, v in ((cache[:, :7], cache[:, :7].contiguous()), (cache[:, :7].contiguous(), cache[:, :7])):
        with pytest.raises(ValueError, match="evenly"):
            kda._attn(q, k, v, None, None)
    for k in (cache, cache[:, :7].contiguous(), cache[:, 9:], cache.transpose(1, 2).contiguous().transpose(1, 2)[:1, :7]):
        _, sizes, p, _, _ = kda._attn(q[:len(k)], k, k, None, None)
        at = {(b, t, h): k[b, t, h].data_ptr() for b in range(len(k)) for t in range(k.shape[1]) for h in range(2)}
        assert all(p[3] + 2 * ((b * k.shape[1] + t) * p[4] + h * p[5]) == x for (b, t, h), x in at.items())
        assert sizes == (len(k), 1, k.shape[1], 4, 2, 64, len(k))
