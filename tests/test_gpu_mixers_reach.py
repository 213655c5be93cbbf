"""How far a NaN in the inputs of causal attention reaches beside the tokens that the formula takes it to.

Tiles are multiplied whole: 64 keys against the 32 rows of a wave in the forward (a key's tile reaches
63 keys further, a row's wave 31 tokens: 94), 32 keys against 128 rows for dq (31 + 127) and 128 keys against
32 rows for dk and dv (127 + 31: 158 both).  Where queries and keys start together their tiles do, too, and
it is less; behind a past they do not.
"""

import pytest
import torch

import test_gpu_attn as at
from test_gpu_around import say

pytestmark = pytest.mark.gpu
FORWARD, BACKWARD = 94, 158
CASES = {  # queries, query and key heads, channels, keys in front of the queries (fewer than them, where negative)
    "no_past": (1, 300, 1, 1, 128, 0), "past": (1, 300, 1, 1, 128, 33), "past_wide": (1, 400, 4, 2, 64, 97),
    "two": (2, 290, 2, 2, 64, 31), "past_odd_group": (1, 260, 6, 2, 128, 1), "fewer_keys": (1, 333, 2, 1, 64, -45),
    "few_queries": (1, 30, 1, 1, 128, 333), "split_rows": (1, 1100, 6, 2, 64, 65),
}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def spoilt(c, name, row, head):
    t = c[name].clone()
    t[0, row, head] = float("nan")
    return dict(c, **{name: t})


def rows(c, name):
    """Keys to spoil: at the edges of tiles of keys, of rows, and of both."""
    B, Tk = c["k"].shape[:2]
    past = Tk - c["q"].shape[1]
    return sorted({r for e in (0, 31, 32, 63, 64, 127, 128, 160, 200, 255, 256) for r in (e, e + past) if 0 <= r < Tk})


@pytest.mark.parametrize("name", CASES)
def test_a_nan_in_a_value_reaches_few_earlier_queries(name):
    say("reach of v", name)
    c = at.case(500 + list(CASES).index(name), *CASES[name])
    Tq, Hq, Hk = c["q"].shape[1], c["q"].shape[2], c["k"].shape[2]
    past, G = c["k"].shape[1] - Tq, Hq // Hk
    out, lse = at.fwd(c)
    for j in rows(c, "v"):
        o, s = at.fwd(spoilt(c, "v", j, 0))
        assert torch.equal(s, lse) and torch.equal(o[1:], out[1:]) and torch.equal(o[:, :, G:], out[:, :, G:])
        sees, clear = max(0, j - past), max(0, j - past - FORWARD)  # the first query that sees it; the first it may reach
        assert torch.isnan(o[0, sees:, :G].float()).all(), j
        assert torch.equal(o[0, :clear], out[0, :clear]), j


@pytest.mark.parametrize("name", CASES)
def test_a_nan_in_a_key_reaches_no_earlier_query(name):
    """Scores that the mask takes are replaced, not weighted: the forward is exact here."""
    say("reach of k", name)
    c = at.case(520 + list(CASES).index(name), *CASES[name])
    Tq, Hq, Hk = c["q"].shape[1], c["q"].shape[2], c["k"].shape[2]
    past, G = c["k"].shape[1] - Tq, Hq // Hk
    out, lse = at.fwd(c)
    for j in rows(c, "k"):
        o, s = at.fwd(spoilt(c, "k", j, 0))
        sees = max(0, j - past)
        assert torch.isnan(s[0, sees:, :G]).all() and torch.isnan(o[0, sees:, :G].float()).all(), j
        assert torch.equal(o[0, :sees], out[0, :sees]) and torch.equal(s[0, :sees], lse[0, :sees]), j
        assert torch.equal(o[1:], out[1:]) and torch.equal(o[:, :, G:], out[:, :, G:])


@pytest.mark.parametrize("name", CASES)
def test_what_a_nan_reaches_in_gradients_behind_a_past(name):
    say("reach in gradients", name)
    c = at.case(540 + list(CASES).index(name), *CASES[name])
    B, Tq, Hq = c["q"].shape[:3]
    Tk, Hk = c["k"].shape[1:3]
    past, G = Tk - Tq, Hq // Hk
    clean = at.bwd(c)
    same = lambda got, cut: all(torch.equal(x[cut], y[cut]) for x, y in zip(got, clean))  # noqa: E731
    for i in sorted({r for e in (0, 31, 32, 127, 128, 160, 250) for r in (e, e - past) if 0 <= r < Tq}):
        for n in ("q", "d_out"):
            dq, dk, dv = got = at.bwd(spoilt(c, n, i, 0))
            others = torch.arange(Tq) != i
            assert torch.equal(dq[0][others], clean[0][0][others]) and torch.equal(dq[:, :, 1:], clean[0][:, :, 1:]), (n, i)
            far = max(0, i + past + 1 + BACKWARD)  # the first key that it may not reach
            assert torch.equal(dk[0, far:], clean[1][0, far:]) and torch.equal(dv[0, far:], clean[2][0, far:]), (n, i)
            if i + past >= 0:
                assert torch.isnan(dq[0, i, 0].float()).all() and torch.isnan(dk[0, :i + past + 1, 0].float()).all(), (n, i)
            assert same(got, slice(1, None)) and torch.equal(dk[:, :, 1:], clean[1][:, :, 1:])
    for j in rows(c, "k"):
        for n, reach in (("k", BACKWARD), ("v", FORWARD)):
            dq, dk, dv = got = at.bwd(spoilt(c, n, j, 0))
            clear = max(0, j - past - reach)
            assert torch.equal(dq[0, :clear], clean[0][0, :clear]), (n, j)
            assert same(got, slice(1, None)) and torch.equal(dq[:, :, G:], clean[0][:, :, G:])
            assert torch.equal(dk[:, :, 1:], clean[1][:, :, 1:]) and torch.equal(dv[:, :, 1:], clean[2][:, :, 1:])
