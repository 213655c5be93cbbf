"""The operators around the core where their work is split: many tiles of a slowly forgetting
recurrence, columns handed out by several counters, the longest tiles of the convolution, and more
items than the q/k backward's grid.  Every element is compared with fp64.

Tolerances of the recurrence, to first order, of every element (e = 2^-23, an ulp):

* a decay a = exp(g): g is off relatively by a few ulp (reciprocal, two products, the product in the
  exponent: 12 e covers them) and by what z = exp(A_log) (raw + dt_bias) is off absolutely, 4 e of
  its terms' size; exp adds an ulp, and each row one rounding of a product of decays and one of a sum,
  with a tenth of that where runs and tiles are joined: together under 4 e.  So a row's state
  is off by step = (|g| (12 + 4 exp(A_log) (|raw| + |dt_bias|)) + 4) e of its size, and the error
  obeys the recurrence itself, run on absolute values.
* sums over tokens: 4 rows and 28 runs of a tile in fp32, under 40 roundings of 2^-24; the rest in fp64.
"""

import math
import os
import re

import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd.function import kda_glr
from oracle import around as A
from test_gpu_around import DEV, HALF, TYPES, Rand, conv_run, dev, near, qk_check, say

pytestmark = pytest.mark.gpu
E = 2.0 ** -23
CSRC = os.path.join(os.path.dirname(kda.__file__), "csrc")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------
def slow_case(seed, H, K, lengths, gate, ty, complement, rest=0):
    """Decays that last for thousands of rows, different in every row and channel: `gate` "given" is
    -10^u, u in [-4, -2]; "bias" has dt_bias around -6; "bound" a lower bound of -0.004; "usual" none of them."""
    r, ty = Rand(seed), TYPES[ty]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32)
    T, N = int(cu[-1]) + rest, len(lengths)
    c = dict(x=r(1, T, H, K, dtype=ty), g=r(1, T, H, K), al=r(H, std=0.3), dt=r(H, K, std=0.3), init=r(N, H, K, std=4.0),
             d_out=r(1, T, H, K, dtype=ty), d_fin=r(N, H, K, std=4.0), cu=cu, lb=-5.0, given=gate == "given",
             complement=complement)
    if gate == "given":
        c["g"] = -10.0 ** (-3 + c["g"].clamp(-1, 1))
        c["al"] = c["dt"] = None
    elif gate == "bias":
        c["dt"] = c["dt"] - 6.0
    elif gate == "bound":
        c["lb"] = -0.004
    c["g"] = c["g"].to(ty)
    if rest:
        for n in ("x", "g", "d_out"):
            c[n][:, T - rest:] = float("nan")
    return {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}


def scan(a, u):
    """h_t = a_t h_{t-1} + u_t by doubling, in fp64; a is 0 where a sequence starts."""
    a, h, d = a.clone(), u.clone(), 1
    while d < h.shape[0]:
        h[d:] += a[d:] * h[:-d].clone()
        a[d:] *= a[:-d].clone()
        d *= 2
    return h


def slow_check(c, values, out, fin, got):
    """Forward and gradients against the recurrence in fp64, row by row, on the GPU."""
    cu = c["cu"].tolist()
    L = cu[-1]
    x, g, do = (c[n][0, :L].double() for n in ("x", "g", "d_out"))
    init, d_fin = c["init"].double(), c["d_fin"].double()
    if c["given"]:
        lg, z, ea, zoff, slope = g, torch.zeros_like(g), 1.0, 0.0, torch.ones_like(g)
    else:
        ea = c["al"].double().exp()[:, None]
        z = ea * (g + c["dt"].double())
        s = torch.sigmoid(z)
        lg, slope, zoff = c["lb"] * s, c["lb"] * s * torch.sigmoid(-z) * ea, 4 * E * ea * (g.abs() + c["dt"].double().abs())
    a, b = lg.exp(), -torch.expm1(lg) if c["complement"] else torch.ones_like(lg)
    u = b * x
    h, before, dh = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    wf, wi = init.clone(), d_fin.clone()
    first, last = [], []
    for n, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
        if hi > lo:
            first.append((n, lo)), last.append((n, hi - 1))
        state = wf[n].clone()
        for t in range(lo, hi):
            state = torch.addcmul(u[t], a[t], state, out=h[t])
        before[lo:hi] = torch.cat([init[n][None], h[lo:hi - 1]]) if hi > lo else before[lo:hi]
        wf[n] = state
        down = wi[n].clone()
        for t in reversed(range(lo, hi)):
            torch.add(do[t], down, out=dh[t])
            down = a[t] * dh[t]
        wi[n] = down
    # the same on absolute values, and the errors that they admit
    step = (lg.abs() * (12 * E + zoff) + 4 * E)
    fn, fr = (torch.tensor(v, device=DEV) for v in zip(*first))
    ln, lr = (torch.tensor(v, device=DEV) for v in zip(*last))
    ar, al_ = a.clone(), torch.cat([a[1:], a[:1]])  # decay into row t from the left, and from the right
    ar[fr], al_[lr] = 0.0, 0.0
    ua = u.abs()
    ua[fr] += a[fr] * init[fn].abs()
    size = scan(ar, ua)
    err = scan(ar, step * size)
    da = do.abs()
    da[lr] += d_fin[ln].abs()
    dsize = scan(al_.flip(0), da.flip(0)).flip(0)
    derr = scan(al_.flip(0), ((torch.cat([step[1:], step[:1]]) + E) * dsize).flip(0)).flip(0)
    prev, perr = torch.cat([size[:1], size[:-1]]), torch.cat([err[:1], err[:-1]])
    prev[fr], perr[fr] = init[fn].abs(), 0.0
    half = HALF[c["x"].dtype]
    own = lambda t, i, w: torch.zeros_like(w).index_copy_(0, i, t)  # noqa: E731
    check = lambda name, v, want, tol, r: near(name, v, want.cpu(), (tol + r * want.abs()).cpu())  # noqa: E731
    check("out", out[0, :L], h, err, half)
    check("final", fin, wf, own(err[lr], ln, wf), 2.0 ** -24)
    check("d_init", got["init"], wi, own(a[fr] * (derr + step * dsize)[fr], fn, wi), 2.0 ** -24)
    check("dx", got["x"][0, :L], dh * b, b * (derr + 16 * E * dsize), half)
    p = before - x if c["complement"] else before
    pa = prev + (x.abs() if c["complement"] else 0)
    draw = dh * a * p * slope
    # the slope is off like the gate: by a few ulp and by what z is off
    doff = a * slope.abs() * (derr * pa + dsize * perr + (16 * E + 2 * zoff) * dsize * pa)
    check("dg", got["g"][0, :L], draw, doff, half)
    if not c["given"]:
        dz, ez = dh * a * p * slope / ea, doff / ea
        check("dd", got["dt"], draw.sum(0), (doff + 40 * 2.0 ** -24 * draw.abs()).sum(0), 2.0 ** -24)
        check("dA", got["al"], (dz * z).sum((0, 2)),
              (ez * z.abs() + dz.abs() * (zoff + (4 + 20) * E * z.abs())).sum((0, 2)), 2.0 ** -24)
    # what the gates are for: a state meets the next ones in reach
    if values == "slow":
        assert lg[:L].sum(0).max() / L > -0.01


def slow_run(c):
    leaf = lambda t: None if t is None else t.detach().requires_grad_(True)  # noqa: E731
    leaves = {n: leaf(c[n]) for n in ("x", "g", "al", "dt", "init") if c[n] is not None}
    out, fin = kda_glr(leaves["x"], leaves["g"], leaves.get("al"), leaves.get("dt"), initial_state=leaves["init"],
                       cu_seqlens=c["cu"], gate_given=c["given"], complement=c["complement"], lower_bound=c["lb"])
    return out, fin, dict(zip(leaves, torch.autograd.grad((out, fin), list(leaves.values()), (c["d_out"], c["d_fin"]))))


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("gate", ["given", "bias", "bound"])
def test_glr_states_that_last_over_many_tiles(gate, complement, ty):
    """43 tiles of 224 rows (86 of 112) in one column, two resets: what enters a tile is the product of the
    maps of many before it, in order.  Four runs have the same bits, however far their searches went."""
    say("slow", gate, complement, ty)
    c = slow_case(80, 1, 64, [9410, 0, 130, 95], gate, ty, complement)
    out, fin, got = slow_run(c)
    for _ in range(3):
        o2, f2, g2 = slow_run(c)
        assert torch.equal(out, o2) and torch.equal(fin, f2) and all(torch.equal(got[n], g2[n]) for n in got)
    slow_check(c, "slow", out, fin, got)


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["bias", "usual"])
@pytest.mark.parametrize("H,K", [(2, 128), (4, 128), (8, 128), (3, 64), (12, 64)])
def test_glr_columns_of_every_counter(H, K, gate, ty):
    """4, 8, 16, 3 and 12 column blocks of 64 channels: columns in four sets, eight sets of one and of two,
    one, and four of three, with many tiles of each and sequences cut anywhere."""
    say("columns", H, K, gate, ty)
    c = slow_case(81, H, K, [4000, 3, 225, 0, 2777, 112, 1], gate, ty, gate == "usual", rest=40)
    out, fin, got = slow_run(c)
    slow_check(c, gate, out, fin, got)
    assert not out[0, -40:].any() and not got["x"][0, -40:].any() and not got["g"][0, -40:].any()


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------
def tile_rows(rule, T, groups):
    """Rows of a tile by the rule of the given name in the source, read there."""
    with open(os.path.join(CSRC, "kda_conv.hip")) as f:
        m = re.search(rf"{rule}\{{(\d+), (\d+), (\d+) \* 1024\}}", f.read())
    r, least, threads = int(m[1]), int(m[2]), int(m[3]) * 1024
    while r > least and math.ceil(T / r) * groups < threads:
        r //= 2
    return r


@pytest.mark.parametrize("ty,lengths,C,rows", [("bf16", [63, 1, 65, 0, 2, 3000, 127, 4960], 16384, 64),
                                               ("bf16", [31, 1, 33, 0, 2, 3000, 1040], 16384, 32),
                                               ("fp32", [63, 1, 65, 0, 2, 3000, 989], 16384, 64)])
def test_conv_walks_its_longest_tiles(ty, lengths, C, rows):
    """Forward tiles of 64 and 32 rows, backward tiles of 128, with sequences that end and start inside
    them and at their edges; a few channels, each of which stands alone, against the oracle."""
    T, W, N, dt = sum(lengths), 4, len(lengths), TYPES[ty]
    say("conv tiles", ty, T, C)
    assert tile_rows("kFwdRule", T, C // (8 if ty == "bf16" else 4)) == rows and tile_rows("kBwdRule", T, C // 4) == 128
    gen = torch.Generator(device=DEV).manual_seed(82)
    r = lambda *s, std=1.0, dtype=torch.float32: (torch.randn(*s, generator=gen, device=DEV) * std).to(dtype)  # noqa: E731
    cu = [0, *torch.tensor(lengths).cumsum(0).tolist()]
    c = dict(x=r(1, T, C, dtype=dt), w=r(C, W, std=0.7), b=r(C, std=0.3), init=r(N, W - 1, C, dtype=dt),
             cu=torch.tensor(cu, dtype=torch.int32), d_out=r(1, T, C, dtype=dt), d_fin=r(N, W - 1, C, dtype=dt), silu=True)
    out, fin, got = conv_run(c)
    cols = torch.tensor([0, 7, C // 2 + 3, C - 1], device=DEV)
    pick = lambda t: t.detach()[..., cols].cpu()  # noqa: E731
    leaves = [pick(c["x"]), c["w"][cols].cpu(), c["b"][cols].cpu(), pick(c["init"])]
    cots = [pick(c["d_out"]), pick(c["d_fin"])]
    (o, f), g = A.grads(lambda x, w, b, i: A.conv(x, w, b, i, cu, True), leaves, cots)
    # sizes as in the small cases: the same problem on absolute values without the activation
    (z, _), gm = A.grads(lambda x, w, b, i: A.conv(x, w, b, i, cu, False), [t.abs() for t in leaves], [t.abs() for t in cots])
    half, zmax = HALF[dt], 1 + z.abs().max().item()
    near("out", pick(out), o, half * o.abs() + 8 * E * z)
    near("final", pick(fin), f, 0.0)
    near("dx", pick(got["x"]), g[0], half * g[0].abs() + 16 * E * zmax * gm[0])
    # a tap's sum over a tile of 128 rows in fp32: 128 roundings of 2^-24 of the sum of sizes; then fp64
    sums = 16 * E * zmax + 128 * 2.0 ** -24 * 1.1
    near("dw", got["w"][cols], g[1], 2.0 ** -24 * g[1].abs() + sums * gm[1])
    near("db", got["b"][cols], g[2], 2.0 ** -24 * g[2].abs() + sums * gm[2])
    near("di", pick(got["init"]), g[3], half * g[3].abs() + 16 * E * zmax * gm[3])


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("ty", ["bf16", "fp32"])
def test_qk_gradients_of_more_items_than_the_grid_has(ty):
    """2200 tokens of 8 chunks of 4 heads: 17600 items for 1024 workgroups of 16, so that some take a second
    one and carry the weights' sums over."""
    with open(os.path.join(CSRC, "kda_qk.hip")) as f:
        s = f.read()
    blocks, heads, threads = (int(re.search(rf"constexpr \w+ {n} = (\d+);", s)[1]) for n in ("kQkBlocks", "HC", "QT"))
    assert 2200 * math.ceil((24 + 8) / heads) > blocks * threads // (128 // 8)
    qk_check(83, 1, 2200, 24, 8, 128, 128, ty, norm="rms", weights=True, fused=True)
