"""Outputs that are one of the inputs, where another workgroup may still read it: refused on the host,
before any device work (the pointers are never dereferenced)."""

import pytest

import chunked_gated_delta_amd as kda

L = kda._lib
P = [0x100000 * (i + 1) for i in range(16)]  # arrays of their own
INVALID = 1


def glr_fwd(x=P[0], out=P[2], init=P[6], fin=P[7]):
    return L.kda_glr_fwd(x, P[1], out, P[3], 1 << 40, P[4], P[5], -5.0, init, fin, None, None, 1, 300, 2, 8, 1, 0, 0, None)


def glr_bwd(dfin=P[8], dinit=P[9], init=P[10]):
    return L.kda_glr_bwd(P[0], P[1], P[2], P[3], dfin, P[4], P[5], P[6], P[7], dinit, P[11], 1 << 40, P[12], P[13], -5.0, init,
                         None, 1, 300, 2, 8, 1, 0, 0, None)


def conv_fwd(x=P[0], out=P[1], init=P[2], fin=P[3], w=P[4]):
    return L.kda_conv_fwd(x, 16, w, None, out, init, fin, None, 1, 300, 16, 4, 1, 0, 0, None)


def conv_bwd(x=P[0], dout=P[1], dx=P[2], dfin=P[3], dinit=P[4], init=P[5], w=P[6]):
    return L.kda_conv_bwd(x, 16, w, None, dout, dfin, dx, P[7], None, dinit, P[8], 1 << 40, init, None, 1, 300, 16, 4, 1, 0, 0,
                          None)


@pytest.mark.parametrize("call,alias", [
    (glr_fwd, dict(init=P[6], fin=P[6])), (glr_bwd, dict(dfin=P[8], dinit=P[8])), (glr_bwd, dict(init=P[10], dinit=P[10])),
    (conv_fwd, dict(x=P[0], out=P[0])), (conv_fwd, dict(init=P[2], fin=P[2])),
    (conv_bwd, dict(x=P[0], dx=P[0])), (conv_bwd, dict(dout=P[1], dx=P[1])), (conv_bwd, dict(dfin=P[3], dinit=P[3])),
    (conv_bwd, dict(init=P[5], dinit=P[5]))])
def test_an_output_that_is_an_input_is_refused(call, alias):
    assert call(**alias) == INVALID
