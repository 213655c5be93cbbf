"""Sizes at the limits of what one call of a token mixer takes (CPU only: every call here is rejected before any
device work, so its pointers are never dereferenced)."""

import pytest

from test_boundary_mixers import INVALID, P, at_bwd, at_fwd, la_bwd, la_fwd, la_step

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
