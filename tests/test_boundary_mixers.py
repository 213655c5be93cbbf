"""Host-side checks of the token mixers beside the core (CPU only: every call here is rejected before any
device work, so its pointers are never dereferenced)."""

import ctypes

import pytest
import torch

import chunked_gated_delta_amd as kda

P = [0x100000 * (i + 1) for i in range(20)]  # arrays of their own
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
NAN, INF = float("nan"), float("inf")
L = kda._lib
QKV = dict(q=P[0], qs=128, qh=64, k=P[1], ks=128, kh=64, v=P[2], vs=128, vh=64)
LA_SIZES = dict(B=1, T=8, H=2, K=64, V=64, N=1)
AT_SIZES = dict(B=1, Tq=8, Tk=8, Hq=2, Hk=2, D=64, N=1)


def la_fwd(**o):
    a = QKV | dict(g=P[3], scale=1.0, out=P[4], ws=P[5], size=1 << 50, init=None, fin=None, cu=None) | LA_SIZES | dict(flags=0)
    assert set(o) <= set(a)
    return L.kda_la_fwd(*(a | o).values(), None)


def la_bwd(**o):
    a = QKV | dict(g=P[3], scale=1.0, dout=P[4], dfin=None, dq=P[5], dk=P[6], dv=P[7], dg=None, di=None, ws=P[8],
                   size=1 << 50, init=None, cu=None) | LA_SIZES | dict(flags=0)
    assert set(o) <= set(a)
    return L.kda_la_bwd(*(a | o).values(), None)


def la_step(**o):
    a = QKV | dict(g=P[3], scale=1.0, out=P[4], init=None, fin=None) | {n: v for n, v in LA_SIZES.items() if n != "N"}
    assert set(o) <= set(a)
    return L.kda_la_step(*(a | o).values(), None)


def at_fwd(**o):
    a = QKV | dict(scale=1.0, out=P[3], lo=None, lse=P[4], ws=P[5], size=1 << 50, cq=None, ck=None) | AT_SIZES | dict(flags=0)
    assert set(o) <= set(a)
    return L.kda_attn_fwd(*(a | o).values(), None)


def at_bwd(**o):
    a = QKV | dict(scale=1.0, out=P[3], lo=P[4], lse=P[5], dout=P[6], dlse=None, dq=P[7], dk=P[8], dv=P[9], ws=P[10],
                   size=1 << 50, cq=None, ck=None) | AT_SIZES | dict(flags=0)
    assert set(o) <= set(a)
    return L.kda_attn_bwd(*(a | o).values(), None)


LA, AT = (la_fwd, la_bwd), (at_fwd, at_bwd)
REFUSED = [
    *[(f, {n: None}, INVALID) for f, names in ((la_fwd, "q k v g out"), (la_bwd, "q k v g dout dq dk dv"), (la_step, "q k v g out"),
                                              (at_fwd, "q k v out lse"), (at_bwd, "q k v out lo lse dout dq dk dv"))
      for n in names.split()],
    *[(f, {n: P[19] + 8}, INVALID) for f, names in ((la_fwd, "q k v out ws init fin"), (la_bwd, "q k v dout dfin dq dk dv di ws init"),
                                                   (la_step, "q k v out init fin"), (at_fwd, "q k v out lo ws"),
                                                   (at_bwd, "q k v out lo dout dq dk dv ws")) for n in names.split()],
    *[(f, {n: P[19] + 2}, INVALID) for f, names in ((la_fwd, "g"), (la_bwd, "g dg"), (at_fwd, "lse"), (at_bwd, "lse dlse"))
      for n in names.split()],
    *[(f, {n: x}, INVALID) for f in (*LA, la_step, *AT) for n in ("qs", "ks", "vs", "qh", "kh", "vh") for x in (-8, 4, 1, (1 << 23) + 8)],
    *[(f, o, INVALID) for f in LA for o in
      (dict(B=0), dict(T=-1), dict(H=0), dict(K=0), dict(V=-64), dict(N=0), dict(N=2), dict(B=2, N=2, cu=P[18]),
       dict(B=2), dict(flags=1), dict(flags=4096), dict(T=1 << 45), dict(B=1 << 40, N=1 << 40, T=1 << 40), dict(H=1 << 40),
       dict(T=1 << 31, cu=P[18]), dict(N=1 << 31, cu=P[18]), dict(scale=NAN), dict(scale=INF))],
    *[(la_step, o, INVALID) for o in (dict(B=0), dict(T=-1), dict(H=0), dict(T=(1 << 20) + 1), dict(B=1 << 30, H=1 << 10),
                                      dict(scale=NAN))],
    *[(f, o, UNSUPPORTED) for f in (*LA, la_step) for o in (dict(K=32), dict(V=96), dict(K=256), dict(K=65))],
    *[(f, o, INVALID) for f in AT for o in
      (dict(B=0), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hk=0), dict(Hq=3), dict(Hk=4), dict(N=0), dict(N=2), dict(B=2),
       dict(cq=P[18]), dict(ck=P[18]), dict(B=2, N=2, cq=P[18], ck=P[18]), dict(flags=1), dict(flags=4096), dict(Tq=1 << 31),
       dict(Tk=1 << 31), dict(Hq=1 << 17), dict(B=1 << 40, N=1 << 40), dict(N=1 << 31, cq=P[18], ck=P[18]), dict(scale=0.0),
       dict(scale=-1.0), dict(scale=NAN), dict(scale=INF))],
    # a group's heads too far apart for 32-bit offsets
    *[(f, o, INVALID) for f in AT for o in (dict(Hq=256, qh=1 << 23), dict(Hq=254, qh=1 << 23, qs=1 << 18))],
    *[(f, o, UNSUPPORTED) for f in AT for o in (dict(D=32), dict(D=96), dict(D=256))],
    *[(f, o, WORKSPACE) for f in (la_bwd, at_bwd) for o in (dict(ws=None), dict(size=63))],
    *[(la_fwd, dict(T=4096) | o, WORKSPACE) for o in (dict(ws=None), dict(size=1 << 16))],
    (at_fwd, dict(ws=None, Tq=1, Tk=4096, B=64, N=64), WORKSPACE),
    (at_fwd, dict(size=1 << 16, Tq=1, Tk=4096, B=64, N=64), WORKSPACE),  # parts of the keys need room
    (la_bwd, dict(size=1 << 20, T=4096, dg=P[12]), WORKSPACE),
    # an output that is an input, or another output
    *[(la_fwd, {"out": P[i]}, INVALID) for i in range(3)], (la_fwd, dict(init=P[9], fin=P[9]), INVALID),
    *[(la_step, {"out": P[i]}, INVALID) for i in range(3)],
    *[(la_bwd, {n: x}, INVALID) for n in ("dq", "dk", "dv") for x in (P[0], P[1], P[2], P[4])], (la_bwd, dict(dk=P[5]), INVALID),
    (la_bwd, dict(dv=P[5]), INVALID), (la_bwd, dict(dv=P[6]), INVALID), (la_bwd, dict(dfin=P[9], di=P[9]), INVALID),
    (la_bwd, dict(init=P[9], di=P[9]), INVALID), (la_bwd, dict(dg=P[3]), INVALID),
    *[(at_fwd, {n: P[i]}, INVALID) for n in ("out", "lo") for i in range(3)], (at_fwd, dict(lo=P[3]), INVALID),
    *[(at_bwd, {n: x}, INVALID) for n in ("dq", "dk", "dv") for x in (P[0], P[1], P[2], P[3], P[4], P[6])],
    (at_bwd, dict(dk=P[7]), INVALID), (at_bwd, dict(dv=P[7]), INVALID), (at_bwd, dict(dv=P[8]), INVALID),
]


@pytest.mark.parametrize("call,change,status", REFUSED)
def test_refused(call, change, status):
    assert call(**change) == status


def test_calls_without_queries_do_nothing():
    """No query: nothing to write, so that arrays without storage will do."""
    assert at_fwd(Tq=0, q=None, out=None, lse=None) == OK == at_fwd(Tq=0, q=None, out=None, lse=None, Hq=254, qh=1 << 23)


@pytest.mark.parametrize("args", [(-1, 2, 64, 64), (8, 0, 64, 64), (8, 2, 32, 64), (8, 2, 64, 65), (1 << 45, 2, 64, 64), (8, 1 << 21, 64, 64)])
def test_sizes_that_no_call_takes_need_no_workspace(args):
    assert kda.kda_la_workspace_size(*args) == 0 and kda.kda_la_bwd_workspace_size(*args, 1) == 0


@pytest.mark.parametrize("args", [(-1, 8, 2, 2, 64, 1), (8, -1, 2, 2, 64, 1), (8, 8, 0, 2, 64, 1), (8, 8, 3, 2, 64, 1), (8, 8, 2, 2, 96, 1),
                                  (8, 8, 2, 2, 64, 0), (1 << 45, 8, 2, 2, 64, 1)])
def test_attention_sizes_that_no_call_takes(args):
    assert kda.kda_attn_workspace_size(*args) == 0 == kda.kda_attn_bwd_workspace_size(*args)


def test_workspaces_are_bounded():
    """States of at most 2048 pieces of a call, and none of a short one; parts of split keys only for few rows."""
    for T in (1, 4096, 1 << 24):
        for H in (1, 7, 96, 200):
            assert kda.kda_la_workspace_size(T, H, 128, 128) <= min(2048, T // 128 * H) * 65536
            assert kda.kda_la_bwd_workspace_size(T, H, 128, 128, 4) <= 256 + 4 * min(2048, T // 128 * H) * 65536 + \
                4 * (4 * H * 2 + 2048) + 256
    assert kda.kda_la_workspace_size(384, 1, 128, 128) == 0 == kda.kda_attn_workspace_size(16384, 16384, 32, 8, 128, 1)
    assert 0 < kda.kda_attn_workspace_size(64, 64 * 8192, 32, 8, 128, 64) <= 64 * 64 * 32 * 129 * 4 + 256
    assert kda.kda_attn_bwd_workspace_size(100, 100, 3, 3, 64, 1) >= 1200
    assert kda.kda_attn_bwd_workspace_size(8194, 8194, 12, 12, 128, 2) <= 512 + 4 * 8194 * 12


def test_the_binding_refuses_tensors_that_are_not_on_the_gpu():
    q, g, ws = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(2), torch.zeros(1024, dtype=torch.uint8)
    for call in (lambda: kda.kda_la_fwd(q, q, q, g, 1.0, q, ws), lambda: kda.kda_la_step(q, q, q, g, 1.0, q),
                 lambda: kda.kda_la_bwd(q, q, q, g, 1.0, q, q, q, q, ws), lambda: kda.kda_attn_fwd(q, q, q, 1.0, q, g, ws),
                 lambda: kda.kda_attn_bwd(q, q, q, 1.0, q, q, g, q, q, q, q, ws)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


class Meta:
    """A _Call whose tensors need not be on a GPU, for the checks behind that one."""

    def __init__(self, first, name):
        self.index = first.get_device()

    token, option = kda._Call.token, kda._Call.option


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(1, 4, 2, 64)), "bfloat16"), (dict(k=torch.zeros(1, 4, 2, 64, dtype=torch.float16)), "bfloat16"),
    (dict(k=torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16)), "shape"), (dict(v=torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16)), "shape"),
    (dict(g=torch.zeros(3)), "shape"), (dict(g=torch.zeros(2, dtype=torch.float64)), "float32"),
    (dict(q=torch.zeros(1, 4, 64, 2, dtype=torch.bfloat16).transpose(2, 3)), "contiguous"), (dict(q=torch.zeros(4, 2, 64)), "must be")])
def test_the_binding_checks_linear_attentions_tensors(change, match, monkeypatch):
    monkeypatch.setattr(kda, "_Call", Meta)
    bf = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    a = dict(q=bf, k=bf, v=bf, g=torch.zeros(2)) | change
    with pytest.raises(ValueError, match=match):
        kda._la(*a.values())


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(1, 4, 2, 64)), "bfloat16"), (dict(k=torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)), "shape"),
    (dict(v=torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16)), "shape"), (dict(cq=torch.zeros(2, dtype=torch.int32)), "together"),
    (dict(cq=torch.zeros(2, dtype=torch.int32), ck=torch.zeros(3, dtype=torch.int32)), "same length"),
    (dict(cq=torch.zeros(2, dtype=torch.int64), ck=torch.zeros(2, dtype=torch.int64)), "int32")])
def test_the_binding_checks_attentions_tensors(change, match, monkeypatch):
    monkeypatch.setattr(kda, "_Call", Meta)
    bf = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    a = dict(q=bf, k=bf, v=bf, cq=None, ck=None) | change
    with pytest.raises(ValueError, match=match):
        kda._attn(*a.values())


def test_tokens_must_lie_evenly_apart(monkeypatch):
    monkeypatch.setattr(kda, "_Call", Meta)
    q = torch.zeros(2, 6, 2, 64, dtype=torch.bfloat16)[:, :4]  # two sequences with a gap between them
    with pytest.raises(ValueError, match="evenly"):
        kda._la(q, q, q, torch.zeros(2))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
