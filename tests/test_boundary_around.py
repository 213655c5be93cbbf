"""Host-side checks of the operators around the core (CPU only: every call here is rejected before
any device work, so its pointers are never dereferenced)."""

import ctypes

import pytest
import torch

import chunked_gated_delta_amd as kda

P, F = 0x1000, 1e-6
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
L = kda._lib


def glr_fwd(**o):
    a = dict(x=P, g=P, out=P, ws=P, size=1 << 40, al=P, dt=P, lb=-5.0, init=None, fin=None, states=None, cu=None, B=1,
             T=8, H=2, K=8, N=1, ty=0, flags=0) | o
    return L.kda_glr_fwd(*a.values(), None)


def glr_bwd(**o):
    a = dict(x=P, g=P, states=P, dout=P, dfin=None, dx=P, dg=P, dA=P, dd=P, dinit=None, ws=P, size=1 << 40, al=P, dt=P,
             lb=-5.0, init=None, cu=None, B=1, T=8, H=2, K=8, N=1, ty=0, flags=0) | o
    return L.kda_glr_bwd(*a.values(), None)


def glr_step(**o):
    a = dict(x=P, g=P, out=P, al=P, dt=P, lb=-5.0, init=None, fin=None, B=1, T=1, H=2, K=8, ty=0, flags=0) | o
    return L.kda_glr_step(*a.values(), None)


def conv_fwd(**o):
    a = dict(x=P, xs=16, w=P, b=None, out=P, init=None, fin=None, cu=None, B=1, T=8, C=16, W=4, N=1, ty=0, flags=0) | o
    return L.kda_conv_fwd(*a.values(), None)


def conv_bwd(**o):
    a = dict(x=P, xs=16, w=P, b=None, dout=P, dfin=None, dx=P, dw=P, db=None, dinit=None, ws=P, size=1 << 40, init=None,
             cu=None, B=1, T=8, C=16, W=4, N=1, ty=0, flags=0) | o
    return L.kda_conv_bwd(*a.values(), None)


def conv_step(**o):
    a = dict(x=P, xs=16, w=P, b=None, out=P, init=None, fin=None, B=1, T=1, C=16, W=4, ty=0, flags=0) | o
    return L.kda_conv_step(*a.values(), None)


def rope_fwd(**o):
    a = dict(q=P, qs=32, qh=16, k=P, ks=16, kh=16, qo=P, ko=P, qw=None, kw=None, pos=P, f=P, eps=F, n=4, Hq=2, Hk=1,
             D=16, R=8, ty=0, flags=0) | o
    return L.kda_qk_rope_fwd(*a.values(), None)


def rope_bwd(**o):
    a = dict(q=P, qs=32, qh=16, k=P, ks=16, kh=16, dqo=P, dko=P, dq=P, dk=P, dqw=None, dkw=None, ws=None, size=0, qw=None,
             kw=None, pos=P, f=P, eps=F, n=4, Hq=2, Hk=1, D=16, R=8, ty=0, flags=0) | o
    return L.kda_qk_rope_bwd(*a.values(), None)


NAN = float("nan")
REFUSED = [
    *[(glr_fwd, {f: None}, INVALID) for f in ("x", "g", "out", "al", "dt")],
    *[(glr_bwd, {f: None}, INVALID) for f in ("x", "g", "states", "dout", "dx", "dg", "dA", "dd", "al", "dt")],
    *[(glr_step, {f: None}, INVALID) for f in ("x", "g", "out", "al", "dt")],
    *[(f, o, INVALID) for f in (glr_fwd, glr_bwd) for o in
      (dict(B=0), dict(T=-1), dict(H=0), dict(K=0), dict(N=0), dict(N=2), dict(B=2, N=2, cu=P), dict(flags=2),
       dict(flags=4096), dict(T=1 << 45), dict(B=1 << 40, N=1 << 40, T=1 << 40), dict(H=1 << 40), dict(T=1 << 31, cu=P),
       dict(H=1 << 15, K=128), dict(x=P + 2), dict(dt=P + 4), dict(init=P + 4), dict(states=P + 8))],
    *[(f, o, UNSUPPORTED) for f in (glr_fwd, glr_bwd, glr_step) for o in
      (dict(K=6), dict(ty=2), dict(ty=-1), dict(lb=-5.5), dict(lb=0.5), dict(lb=NAN))],
    *[(f, o, WORKSPACE) for f in (glr_fwd, glr_bwd) for o in (dict(ws=None), dict(size=256))],
    (glr_step, dict(flags=2048), INVALID), (glr_step, dict(B=0), INVALID), (glr_step, dict(out=P + 4), INVALID),
    *[(conv_fwd, {f: None}, INVALID) for f in ("x", "w", "out")],
    *[(conv_bwd, {f: None}, INVALID) for f in ("x", "w", "dout", "dx", "dw")],
    *[(conv_step, {f: None}, INVALID) for f in ("x", "w", "out")],
    *[(f, o, INVALID) for f in (conv_fwd, conv_bwd) for o in
      (dict(B=0), dict(T=-1), dict(C=0), dict(N=0), dict(N=2), dict(B=2, N=2, cu=P), dict(flags=128), dict(xs=8),
       dict(xs=18), dict(x=P + 2), dict(init=P + 2), dict(w=P + 8), dict(b=P + 4), dict(T=1 << 50), dict(T=1 << 31, cu=P))],
    *[(f, o, UNSUPPORTED) for f in (conv_fwd, conv_bwd, conv_step) for o in
      (dict(C=12), dict(W=5), dict(W=1), dict(ty=7))],
    (conv_bwd, dict(ws=None), WORKSPACE), (conv_bwd, dict(size=16), WORKSPACE), (conv_step, dict(flags=2048), INVALID),
    *[(rope_fwd, {f: None}, INVALID) for f in ("q", "k", "qo", "ko", "pos", "f")],
    *[(rope_bwd, {f: None}, INVALID) for f in ("q", "k", "dqo", "dko", "dq", "dk", "pos", "f")],
    *[(f, o, INVALID) for f in (rope_fwd, rope_bwd) for o in
      (dict(n=-1), dict(Hq=0, Hk=0), dict(Hq=-1), dict(D=0), dict(R=24), dict(eps=NAN), dict(eps=-1.0), dict(flags=1),
       dict(flags=4 | 512), dict(qs=8), dict(qs=34), dict(qh=8), dict(ks=-16), dict(q=P + 2), dict(k=P + 4),
       dict(n=1 << 60))],
    *[(f, o, UNSUPPORTED) for f in (rope_fwd, rope_bwd) for o in (dict(D=20), dict(D=520, qh=520, qs=1040, ks=520, kh=520), dict(R=4), dict(ty=3))],
    (rope_fwd, dict(qs=16), INVALID), (rope_fwd, dict(Hk=2, ks=16), INVALID),  # in place over rows that overlap
    (rope_bwd, dict(dqw=P), WORKSPACE), (rope_bwd, dict(dkw=P, ws=P, size=64), WORKSPACE),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refused(i):
    f, o, want = REFUSED[i]
    assert f(**o) == want, (f.__name__, o)


def test_sizes():
    assert kda.kda_glr_workspace_size(0, 1, 4) > 0 and kda.kda_glr_workspace_size(8, 0, 4) == 0
    assert kda.kda_glr_bwd_workspace_size(4096, 8, 128) >= kda.kda_glr_workspace_size(4096, 8, 128)
    assert kda.kda_glr_states_size(4096, 8, 128) >= 4096 // 128 * 8 * 128 * 4
    assert kda.kda_glr_states_size(1 << 60, 1 << 20, 128) == 0
    assert kda.kda_conv_bwd_workspace_size(100, 16, 4) > 0 and kda.kda_conv_bwd_workspace_size(100, 16, 5) == 0
    assert kda.kda_qk_rope_bwd_workspace_size(0, 1, 0, 64) > 0 and kda.kda_qk_rope_bwd_workspace_size(4, 1, 1, 60) == 0
    # a size bought for an upper bound on the tokens serves every smaller call
    for size in (lambda t: kda.kda_glr_workspace_size(t, 3, 64), lambda t: kda.kda_glr_bwd_workspace_size(t, 3, 64),
                 lambda t: kda.kda_glr_states_size(t, 3, 64), lambda t: kda.kda_conv_bwd_workspace_size(t, 4096, 4)):
        got = [size(t) for t in range(0, 40000, 37)]
        assert all(a <= b for a, b in zip(got, got[1:]))


def test_flags_do_not_collide():
    flags = [getattr(kda, n) for n in dir(kda) if n.startswith("FLAG_")]
    assert len(set(flags)) == len(flags) and all(f & (f - 1) == 0 for f in flags)


def test_the_core_refuses_the_new_flags():
    """The bits of these operators are none of kda_fwd_ex's."""
    for f in (kda.FLAG_COMPLEMENT, kda.FLAG_SILU, kda.FLAG_RMS_NORM, kda.FLAG_INTERLEAVED, kda.FLAG_ZERO_REST):
        assert L.kda_fwd_ex(P, P, P, P, P, ctypes.c_float(0.1), P, P, 1 << 40, P, P, ctypes.c_float(-5.0), None, None,
                            None, 1, 64, 2, 128, 128, 1, f, None) == INVALID


def test_the_binding_rejects_host_tensors():
    from chunked_gated_delta_amd.function import kda_glr, kda_qk_norm_rope, kda_short_conv

    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="device"):
        kda_glr(x, x, torch.zeros(2), torch.zeros(2, 8))
    with pytest.raises(ValueError, match="device"):
        kda_short_conv(x.view(1, 4, 16), torch.zeros(16, 4))
    with pytest.raises(ValueError, match="device"):
        kda_qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="gate_given"):
        kda_glr(x, x, torch.zeros(2), gate_given=True)
    with pytest.raises(ValueError, match="norm"):
        kda_qk_norm_rope(x, x, norm="l1")
