"""The operators around the core on the GPU against their fp64 oracles (oracle/around.py).

Tolerances are bounds of the rounding of fp32 arithmetic, to first order, plus half a step of
the output's type (bf16 2^-8, fp32 2^-24 of the value):

* recurrence: one decay a = exp(g) is off by at most STEP relative (|g| <= 5 formed from an exp2,
  a reciprocal and two products, each within an ulp or two of 2^-23: 5 * 4 ulp, plus the products
  and sums of the recurrence itself), so the state's error obeys the recurrence itself with
  STEP * |state| as its input.  Both that and the state's size are run in fp64 on absolute values.
* convolution: (W + 2) roundings of sum |w| |x|, through an activation of slope below 1.1.
* norm and rotation: sums of at most 512 squares (lane, then tree: < 20 roundings) and a turn
  by sines within 2^-18 (bf16, the hardware's) or 2^-22 (fp32), relative to the pair's size.
"""

import math

import numpy as np
import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd.function import kda_chunk, kda_glr, kda_qk_norm_rope, kda_short_conv
from oracle import around as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = 32 * 2.0 ** -23
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(*a):
    print(*a, flush=True)


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g) * std).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


def near(name, got, want, tol):
    got = got.detach().double().cpu()
    want = want.reshape(got.shape)
    tol = torch.as_tensor(tol, dtype=torch.float64).expand(want.numel()).reshape(want.shape) if not torch.is_tensor(tol) \
        else tol.reshape(want.shape)
    off = (got - want).abs() - tol
    assert not torch.isnan(off).any(), name
    worst = off.max().item() if off.numel() else -1
    assert worst <= 0, (name, worst, ((got - want).abs() / tol.clamp(min=1e-300)).max().item())


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------
def glr_case(seed, B, T, H, K, lengths=None, rest=0, ty="bf16", init=True, given=False, complement=False):
    r, ty = Rand(seed), TYPES[ty]
    cu = None
    if lengths is not None:
        cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32)
        B, T = 1, int(cu[-1]) + rest
    N = B if cu is None else len(lengths)
    c = dict(x=r(B, T, H, K, dtype=ty), g=r(B, T, H, K, std=2.0), al=r(H, std=1.0), dt=r(H, K, std=0.3),
             init=r(N, H, K) if init else None, cu=cu, d_out=r(B, T, H, K, dtype=ty), d_fin=r(N, H, K), given=given,
             complement=complement)
    if given:
        c["g"] = -5 * torch.sigmoid(c["g"])
        c["al"] = c["dt"] = None
    c["g"] = c["g"].to(ty)
    if rest:  # rows behind the last sequence hold nothing that may be used
        for n in ("x", "g", "d_out"):
            c[n][:, T - rest:] = float("nan")
    return c


def glr_oracle(c, grad=True):
    cu = None if c["cu"] is None else c["cu"].tolist()
    f = lambda x, g, al, dt, i: A.glr(x, g, al, dt, -5.0, i, cu, c["given"], c["complement"])  # noqa: E731
    live = lambda t: t.nan_to_num(0.0)  # noqa: E731  (rows of no sequence)
    leaves = [live(c["x"]), live(c["g"]), c["al"], c["dt"], c["init"]]
    if not grad:
        return f(*(A.f64(t) for t in leaves)), None
    return A.grads(f, leaves, [live(c["d_out"]), c["d_fin"]])


def glr_bounds(c):
    """Tolerances without the output rounding: out, final, dx, d_raw, dA, d_dt_bias, d_init."""
    x, g, d_out = (A.f64(c[n].nan_to_num(0.0)) for n in ("x", "g", "d_out"))
    B, T, H, K = x.shape
    x, g, d_out = (t.reshape(B * T, H, K).abs() if t is not g else t.reshape(B * T, H, K) for t in (x, g, d_out))
    if c["given"]:
        lg, slope, z = g, torch.ones_like(g), torch.zeros_like(g)
    else:
        ea = A.f64(c["al"]).exp()[:, None]
        z = ea * (g + A.f64(c["dt"]))
        s = torch.sigmoid(z)
        lg, slope = -5.0 * s, 5.0 * s * (1 - s) * ea
    a = lg.exp()
    u = -torch.expm1(lg) * x if c["complement"] else x
    n_seq = B if c["cu"] is None else len(c["cu"]) - 1
    h0 = torch.zeros(n_seq, H, K, dtype=torch.float64) if c["init"] is None else A.f64(c["init"]).abs()
    size, err, prev, perr = (torch.zeros_like(x) for _ in range(4))
    dsize, derr = torch.zeros_like(x), torch.zeros_like(x)
    fin, di = torch.zeros_like(h0), torch.zeros_like(h0)
    for n, (lo, hi) in enumerate(A.bounds(B, T, None if c["cu"] is None else c["cu"].tolist())):
        h, e = h0[n], torch.zeros(H, K, dtype=torch.float64)
        for t in range(lo, hi):
            prev[t], perr[t] = h, e
            e = a[t] * (e + STEP * h) + STEP * u[t]
            h = a[t] * h + u[t]
            size[t], err[t] = h, e
        fin[n] = e
        d, e = A.f64(c["d_fin"])[n].abs(), torch.zeros(H, K, dtype=torch.float64)
        for t in reversed(range(lo, hi)):
            dh = d_out[t] + d
            dsize[t], derr[t] = dh, e + 2.0 ** -23 * dh
            d, e = a[t] * dh, a[t] * (derr[t] + STEP * dh)
        di[n] = e
    b = -torch.expm1(lg) if c["complement"] else torch.ones_like(lg)
    dx = b * (derr + STEP * dsize) + 2.0 ** -126 * dsize
    p = prev + (x if c["complement"] else 0)
    # The gate's slope lb s (1 - s) exp(A_log) is off by another STEP, and by what exp(-z) is off
    # where z is large: z = exp(A_log) raw + exp(A_log) dt_bias carries 4 roundings of 2^-23
    # (exp(A_log), log2(e), the product, the sum) of its terms' size, and exp(-z) is off
    # relatively by as much as z is absolutely.
    # The fp64 oracle's own 1 - s is off by 2^-53, and what is under fp32's smallest normal number
    # (2^-126) may come out as zero.
    tiny = 2.0 ** -126
    oracle = 0.0 if c["given"] else 5 * 2.0 ** -52 * ea
    zoff = 0 if c["given"] else 4 * 2.0 ** -23 * ea * (g.abs() + A.f64(c["dt"]).abs())
    draw = a * slope * (derr * p + dsize * perr + (2 * STEP + zoff) * dsize * p) + (oracle + tiny) * dsize * p
    return dict(out=err, fin=fin, dx=dx, draw=draw, dA=(draw * (z.abs() + zoff) / (1 if c["given"] else ea)).sum((0, 2)),
                dd=draw.sum(0), di=di)


def glr_run(c, **kw):
    leaf = lambda t: None if t is None else t.to(DEV).requires_grad_(True)  # noqa: E731
    x, g, al, dt, i = (leaf(c[n]) for n in ("x", "g", "al", "dt", "init"))
    out, fin = kda_glr(x, g, al, dt, initial_state=i, cu_seqlens=dev(c["cu"]), gate_given=c["given"],
                       complement=c["complement"])
    leaves = [t for t in (x, g, al, dt, i) if t is not None]
    return out, fin, dict(zip([n for n, t in zip(("x", "g", "al", "dt", "init"), (x, g, al, dt, i)) if t is not None],
                              torch.autograd.grad((out, fin), leaves, (dev(c["d_out"]), dev(c["d_fin"])))))


def glr_check(c):
    (o, f), g = glr_oracle(c)
    t = glr_bounds(c)
    out, fin, got = glr_run(c)
    torch.cuda.synchronize()
    half = HALF[c["x"].dtype]
    near("out", out, o, t["out"] + half * o.abs().reshape(t["out"].shape))
    near("final", fin, f, t["fin"] + 2.0 ** -24 * f.abs())
    for name, want, tol, r in (("x", g[0], t["dx"], half), ("g", g[1], t["draw"], half), ("al", g[2], t["dA"], 2.0 ** -24),
                               ("dt", g[3], t["dd"], 2.0 ** -24), ("init", g[4], t["di"], 2.0 ** -24)):
        if want is not None:
            near("d" + name, got[name], want, tol + r * want.abs().reshape(tol.shape))
    return out, fin, got


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,H,K", [(1, 1, 1, 4), (2, 1, 3, 64), (1, 7, 1, 12), (1, 127, 2, 64), (3, 128, 1, 128),
                                     (1, 129, 3, 100), (2, 300, 5, 32), (1, 1000, 1, 128)])
def test_glr_batches(B, T, H, K, ty):
    say("glr", B, T, H, K, ty)
    glr_check(glr_case(1, B, T, H, K, ty=ty, complement=T % 2 == 0, given=T == 7))


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lengths,rest", [([5, 0, 130, 1, 1, 0, 250, 64], 0), ([0, 0, 3], 0), ([128, 128], 37),
                                          ([1] * 140, 200), ([0, 0], 5), ([700], 1)])
def test_glr_packed(lengths, rest, complement, given):
    say("glr packed", lengths, rest, complement, given)
    c = glr_case(2, 1, 0, 2, 68, lengths, rest, complement=complement, given=given)
    out, _, got = glr_check(c)
    if rest:  # fresh memory behind the last sequence comes back as zeros
        assert not out[:, -rest:].any() and not got["x"][:, -rest:].any() and not got["g"][:, -rest:].any()


def test_glr_without_states_and_without_tokens():
    c = glr_case(3, 2, 200, 2, 32, init=False)
    glr_check(c)
    with torch.no_grad():  # the inference call keeps no states: the same bits
        out, fin = kda_glr(dev(c["x"]), dev(c["g"]), dev(c["al"]), dev(c["dt"]))
    o2, f2, _ = glr_run(c)
    assert torch.equal(out, o2) and torch.equal(fin, f2)
    c = glr_case(4, 2, 0, 2, 32)
    out, fin, g = glr_run(c)
    torch.cuda.synchronize()
    assert out.numel() == 0 and torch.equal(fin.cpu(), c["init"]) and torch.equal(g["init"].cpu(), c["d_fin"])
    assert not g["al"].any() and not g["dt"].any()
    c = glr_case(4, 1, 0, 2, 32, lengths=[0, 0, 0])
    out, fin, g = glr_run(c)
    torch.cuda.synchronize()
    assert torch.equal(fin.cpu(), c["init"]) and torch.equal(g["init"].cpu(), c["d_fin"])


def test_glr_keeps_nan_and_infinity_where_they_are():
    """A NaN stays in its sequence and channel; an infinity is dropped by a decay of zero."""
    c = glr_case(5, 1, 0, 2, 64, [100, 60, 240, 100])
    clean = glr_run(c)
    bad = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in c.items()}
    bad["x"][0, 120, 1, 5] = float("nan")
    bad["g"][0, 30, 0, 3] = float("nan")
    bad["x"][0, 200, 0, 7] = float("inf")
    out, fin, got = glr_run(bad)
    hit = torch.zeros_like(c["x"], dtype=torch.bool)
    hit[0, 120:160, 1, 5] = hit[0, 30:100, 0, 3] = hit[0, 200:400, 0, 7] = True
    o, oc = out.detach().cpu(), clean[0].detach().cpu()
    assert torch.equal(o[~hit], oc[~hit]) and not torch.isfinite(o[hit]).any()
    fh = torch.zeros(4, 2, 64, dtype=torch.bool)
    fh[1, 1, 5] = fh[0, 0, 3] = fh[2, 0, 7] = True
    f, fc = fin.detach().cpu(), clean[1].detach().cpu()
    assert torch.equal(f[~fh], fc[~fh]) and not torch.isfinite(f[fh]).any()
    # gradients: other sequences' and channels' are untouched
    other = torch.ones_like(hit)
    other[0, :100, 0, 3] = other[0, 100:160, 1, 5] = other[0, 160:400, 0, 7] = False
    for n in ("x", "g"):
        assert torch.equal(got[n].cpu()[other], clean[2][n].cpu()[other]), n
    # a given decay of minus infinity drops what was before
    x, g = torch.ones(1, 300, 1, 4), torch.zeros(1, 300, 1, 4)
    g[0, 150] = -math.inf
    out, _ = kda_glr(dev(x), dev(g), gate_given=True)
    want = torch.cat([torch.arange(1, 151), torch.arange(1, 151)]).float()
    assert torch.equal(out.cpu()[0, :, 0, 0], want)


def test_glr_c_calls_leave_rows_and_take_no_outputs():
    """Without FLAG_ZERO_REST the rows behind the last sequence stay as they were; final_state,
    d_final and d_initial_state may be absent."""
    c = glr_case(6, 1, 0, 2, 32, [70, 100], rest=90)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}
    T = d["x"].shape[1]
    ws = torch.empty(kda.kda_glr_bwd_workspace_size(T, 2, 32), dtype=torch.uint8, device=DEV)
    st = torch.empty(kda.kda_glr_states_size(T, 2, 32), dtype=torch.uint8, device=DEV)
    out, dx, dg = (torch.full_like(d["x"], 7.0) for _ in range(3))
    dA, dd = torch.empty_like(d["al"]), torch.empty_like(d["dt"])
    kda.kda_glr_fwd(d["x"], d["g"], out, ws, d["al"], d["dt"], -5.0, d["init"], None, st, d["cu"])
    kda.kda_glr_bwd(d["x"], d["g"], st, d["d_out"], dx, dg, dA, dd, ws, d["al"], d["dt"], -5.0, d["init"], None, None,
                    d["cu"])
    torch.cuda.synchronize()
    for t in (out, dx, dg):
        assert (t[:, 170:] == 7.0).all() and not (t[:, :170] == 7.0).all()
    c["d_fin"] = torch.zeros_like(c["d_fin"])
    (o, _), g = glr_oracle(c)
    t = glr_bounds(c)
    near("out", out[:, :170], o[:170], t["out"][:170] + 2.0 ** -8 * o[:170].abs())
    near("dx", dx[:, :170], g[0].reshape(T, 2, 32)[:170], t["dx"][:170] + 2.0 ** -8 * g[0].reshape(T, 2, 32)[:170].abs())
    near("dA", dA, g[2], t["dA"] + 2.0 ** -24 * g[2].abs())


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
def test_glr_step_continues_the_forward(ty):
    c = glr_case(7, 3, 40, 3, 36, ty=ty, complement=True)
    (o, f), _ = glr_oracle(c, grad=False)
    t = glr_bounds(c)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}
    out = torch.empty_like(d["x"])
    with torch.no_grad():
        o1, state = kda_glr(d["x"][:, :37].contiguous(), d["g"][:, :37].contiguous(), d["al"], d["dt"],
                            initial_state=d["init"], complement=True)
    out[:, :37] = o1
    for a, b in ((37, 38), (38, 40)):  # one token, then two, in place
        part = torch.empty(3, b - a, 3, 36, dtype=out.dtype, device=DEV)
        kda.kda_glr_step(d["x"][:, a:b].contiguous(), d["g"][:, a:b].contiguous(), part, d["al"], d["dt"], -5.0, state,
                         state, flags=kda.FLAG_COMPLEMENT)
        out[:, a:b] = part
    near("out", out, o, t["out"] + HALF[c["x"].dtype] * o.abs())
    near("final", state, f, t["fin"] + 2.0 ** -24 * f.abs())


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("H,K", [(1, 4), (3, 128), (5, 64), (7, 192)])
def test_glr_many_tiles_hand_states_on(H, K, ty):
    """More tiles than workgroups run at once, one to 21 columns, sequences that start anywhere: a
    few channels against the fp64 recurrence, and the fault word stays clear."""
    lengths = [3, 20000, 0, 223, 225, 12345, 1]
    say("glr tiles", H, K, ty)
    c = glr_case(30, 1, 0, H, K, lengths, 40, ty=ty, complement=H == 3)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}
    T, N, fl = d["x"].shape[1], len(lengths), kda.FLAG_COMPLEMENT if c["complement"] else 0
    ws = torch.empty(kda.kda_glr_bwd_workspace_size(T, H, K), dtype=torch.uint8, device=DEV).fill_(255)
    st = torch.empty(kda.kda_glr_states_size(T, H, K), dtype=torch.uint8, device=DEV).fill_(255)
    out, dx, dg = (torch.empty_like(d["x"]) for _ in range(3))
    fin, di = torch.empty_like(d["init"]), torch.empty_like(d["init"])
    dA, dd = torch.empty_like(d["al"]), torch.empty_like(d["dt"])
    kda.kda_glr_fwd(d["x"], d["g"], out, ws, d["al"], d["dt"], -5.0, d["init"], fin, st, d["cu"], fl)
    assert kda.kda_workspace_faults(ws) == 0
    kda.kda_glr_bwd(d["x"], d["g"], st, d["d_out"], dx, dg, dA, dd, ws, d["al"], d["dt"], -5.0, d["init"], d["d_fin"],
                    di, d["cu"], fl)
    assert kda.kda_workspace_faults(ws) == 0
    # fp64 on the GPU, rows in a loop, all channels at once
    x, g, do = (t.double()[0].nan_to_num(0.0) for t in (d["x"], d["g"], d["d_out"]))
    z = d["al"].double().exp()[:, None] * (g + d["dt"].double())
    s = torch.sigmoid(z)
    lg = -5.0 * s
    a, b = lg.exp(), -torch.expm1(lg) if fl else torch.ones_like(lg)
    u = b * x
    h, before, dh = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    cu, wf, wi = c["cu"].tolist(), d["init"].double().clone(), d["d_fin"].double().clone()
    for n in range(N):
        state = wf[n].clone()
        for t in range(cu[n], cu[n + 1]):
            before[t] = state
            state = torch.addcmul(u[t], a[t], state, out=h[t])
        wf[n] = state
        down = wi[n].clone()
        for t in reversed(range(cu[n], cu[n + 1])):
            torch.add(do[t], down, out=dh[t])
            down = a[t] * dh[t]
        wi[n] = down
    L = cu[-1]
    p = before - x if fl else before
    draw = dh * a * p * (-5.0 * s * (1 - s)) * d["al"].double().exp()[:, None]
    # an ulp of 2^-23 a row, for as long as a decay lasts: 300 rows at the slowest gates drawn here
    dz = dh * a * p * (-5.0 * s * (1 - s))
    half = HALF[TYPES[ty]]
    for name, got, want, r in (("out", out[0, :L], h[:L], half), ("final", fin, wf, 0), ("d_init", di, wi, 0),
                               ("dx", dx[0, :L], (dh * b)[:L], half), ("dg", dg[0, :L], draw[:L], half),
                               ("dA", dA, (dz * z).sum((0, 2)), 0), ("dd", dd, draw.sum(0), 0)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= r + 300 * 2.0 ** -23, (name, rel)


def test_glr_is_the_same_from_run_to_run():
    c = glr_case(8, 1, 0, 4, 128, [900, 3000, 0, 196])
    runs = [glr_run(c) for _ in range(4)]
    for out, fin, got in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(fin, runs[0][1])
        assert all(torch.equal(got[n], runs[0][2][n]) for n in got)


def test_glr_long_sequence_by_its_parts():
    """16,000 tokens in one call equal the same tokens in pieces that hand the state on, and in fp32
    a constant decay has its closed form to the end."""
    c = glr_case(9, 1, 16000, 1, 128, complement=True)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}
    with torch.no_grad():
        out, fin = kda_glr(d["x"], d["g"], d["al"], d["dt"], initial_state=d["init"], complement=True)
        st, parts = d["init"], []
        for lo in range(0, 16000, 1600):
            o, st = kda_glr(d["x"][:, lo:lo + 1600].contiguous(), d["g"][:, lo:lo + 1600].contiguous(), d["al"],
                            d["dt"], initial_state=st, complement=True)
            parts.append(o)
    # decays here forget within some hundred tokens: 2^-14 of unit-sized states covers both roundings
    assert torch.allclose(fin, st, atol=2.0 ** -14, rtol=2.0 ** -14)
    assert torch.allclose(out.float(), torch.cat(parts, 1).float(), atol=2.0 ** -9, rtol=2.0 ** -7)
    T = 60000
    one = torch.ones(1, T, 1, 4, device=DEV)
    out, _ = kda_glr(one, torch.full_like(one, -1e-4), gate_given=True, complement=True)
    # 1 - exp(-1e-4 t); a decay's rounding of 2^-24 lasts 1e4 tokens: 1e4 * 2^-24, and as much again
    want = -torch.expm1(-1e-4 * torch.arange(1, T + 1, dtype=torch.float64) * float(np.float32(1e-4) / 1e-4))
    assert (out[0, :, 0, 0].double().cpu() - want).abs().max() <= 2e4 * 2.0 ** -24


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------
def conv_case(seed, B, T, C, W, lengths=None, rest=0, ty="bf16", init=True, bias=True, silu=True):
    r, ty = Rand(seed), TYPES[ty]
    cu = None
    if lengths is not None:
        cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32)
        B, T = 1, int(cu[-1]) + rest
    N = B if cu is None else len(lengths)
    c = dict(x=r(B, T, C, dtype=ty), w=r(C, W, std=0.7), b=r(C, std=0.3) if bias else None,
             init=r(N, W - 1, C, dtype=ty) if init else None, cu=cu, d_out=r(B, T, C, dtype=ty),
             d_fin=r(N, W - 1, C, dtype=ty), silu=silu)
    if rest:
        c["x"][:, T - rest:] = c["d_out"][:, T - rest:] = float("nan")
    return c


def conv_run(c, x=None):
    leaf = lambda t: None if t is None else t.to(DEV).requires_grad_(True)  # noqa: E731
    x = leaf(c["x"]) if x is None else x
    w, b, i = (leaf(c[n]) for n in ("w", "b", "init"))
    out, fin = kda_short_conv(x, w, b, silu=c["silu"], initial_state=i, cu_seqlens=dev(c["cu"]))
    names = [n for n, t in zip(("x", "w", "b", "init"), (x, w, b, i)) if t is not None]
    leaves = [t for t in (x, w, b, i) if t is not None]
    return out, fin, dict(zip(names, torch.autograd.grad((out, fin), leaves, (dev(c["d_out"]), dev(c["d_fin"])))))


def conv_check(c, x=None):
    cu = None if c["cu"] is None else c["cu"].tolist()
    live = lambda t: t.nan_to_num(0.0)  # noqa: E731
    leaves = [live(c["x"]), c["w"], c["b"], c["init"]]
    cots = [live(c["d_out"]), c["d_fin"]]
    (o, f), g = A.grads(lambda x, w, b, i: A.conv(x, w, b, i, cu, c["silu"]), leaves, cots)
    # sizes: the same problem on absolute values, without the activation (its slope is below 1.1)
    mag = [None if t is None else t.abs() for t in leaves]
    (zo, _), gm = A.grads(lambda x, w, b, i: A.conv(x, w, b, i, cu, False), mag, [t.abs() for t in cots])
    z = zo  # sum |w| |x|
    half, e = HALF[c["x"].dtype], 2.0 ** -23
    out, fin, got = conv_run(c, x)
    torch.cuda.synchronize()
    near("out", out, o, half * o.abs() + 8 * e * z)
    near("final", fin, f, 0.0)
    # dz is off by 8 e of |dy| (1 + sum |w| |x|); every gradient sums such terms
    zmax = 1 + z.abs().max().item() if z.numel() else 1.0
    for n, want, m, r in (("x", g[0], gm[0], half), ("w", g[1], gm[1], 2.0 ** -24), ("b", g[2], gm[2], 2.0 ** -24),
                          ("init", g[3], gm[3], half)):
        if want is not None:
            near("d" + n, got[n], want, r * want.abs() + 16 * e * zmax * m)
    return out, fin, got


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 8, 4), (4, 1, 24, 2), (2, 2, 8, 4), (2, 3, 16, 3), (1, 67, 40, 4),
                                     (3, 129, 8, 2), (1, 300, 520, 4)])
def test_conv_batches(B, T, C, W, silu, ty):
    say("conv", B, T, C, W, silu, ty)
    conv_check(conv_case(11, B, T, C, W, ty=ty, silu=silu, bias=T % 2 == 1))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lengths,rest", [([5, 0, 130, 1, 2, 0, 3, 64], 0), ([0, 0, 3], 0), ([8, 8, 16, 1], 37),
                                          ([1] * 40, 20), ([0, 0], 5), ([2, 2, 2, 2, 2], 0), ([300], 1)])
def test_conv_packed(lengths, rest, W):
    say("conv packed", lengths, rest, W)
    out, _, got = conv_check(conv_case(12, 1, 0, 16, W, lengths, rest))
    if rest:
        assert not out[:, -rest:].any() and not got["x"][:, -rest:].any()


def test_conv_over_long_tiles():
    """Enough channels that a thread walks its longest tiles (64 rows forward, 128 backward), with
    sequences that end and start inside them and at their edges."""
    c = conv_case(13, 1, 0, 16384, 4, [127, 1, 129, 0, 2, 253, 31, 1600])
    x = c["x"]
    out, fin, got = conv_run(c)
    near_cols = slice(0, 16384, 4001)  # a few channels against the oracle: each stands alone
    part = {k: (v[..., near_cols].contiguous() if k in ("x", "init", "d_out", "d_fin") else v) for k, v in c.items()}
    part["w"], part["b"] = c["w"][near_cols].contiguous(), c["b"][near_cols].contiguous()
    cu = c["cu"].tolist()
    (o, f), g = A.grads(lambda x, w, b, i: A.conv(x, w, b, i, cu, True), [part[n] for n in ("x", "w", "b", "init")],
                        [part["d_out"], part["d_fin"]])
    e = 2.0 ** -23
    near("out", out[..., near_cols], o, 2.0 ** -8 * o.abs() + 200 * e)
    near("final", fin[..., near_cols], f, 0.0)
    near("dx", got["x"][..., near_cols], g[0], 2.0 ** -8 * g[0].abs() + 2000 * e)
    near("dw", got["w"][near_cols], g[1], 2.0 ** -24 * g[1].abs() + 2200 * 64 * e)
    near("db", got["b"][near_cols], g[2], 2.0 ** -24 * g[2].abs() + 2200 * 64 * e)
    near("di", got["init"][..., near_cols], g[3], 2.0 ** -8 * g[3].abs() + 2000 * e)
    assert x.shape[1] == 2143


def test_conv_takes_a_slice_of_a_projection():
    c = conv_case(14, 3, 50, 24, 4)
    wide = torch.full((3, 50, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[..., 16:40] = dev(c["x"])
    conv_check(c, wide[..., 16:40].detach().requires_grad_(True))
    with pytest.raises(ValueError, match="evenly"):
        kda_short_conv(wide[:, :20, 16:40], dev(c["w"]))


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_step_continues_the_forward(ty, W):
    c = conv_case(15, 5, 12, 40, W, ty=ty)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in c.items()}
    with torch.no_grad():
        want, fin = kda_short_conv(d["x"], d["w"], d["b"], initial_state=d["init"])
        out, st = kda_short_conv(d["x"][:, :7].contiguous(), d["w"], d["b"], initial_state=d["init"])
    parts = [out]
    for a, b in ((7, 8), (8, 9), (9, 12)):
        part = torch.empty(5, b - a, 40, dtype=out.dtype, device=DEV)
        x = d["x"][:, a:b] if b - a == 1 else d["x"][:, a:b].contiguous()
        kda.kda_conv_step(x, d["w"], part, d["b"], st, st, flags=kda.FLAG_SILU)
        parts.append(part)
    assert torch.equal(torch.cat(parts, 1), want) and torch.equal(st, fin)  # the same sums in the same order


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
def qk_check(seed, B, T, Hq, Hk, D, R, ty="bf16", norm="l2", inter=False, weights=False, far=0, fused=False):
    say("qk", B, T, Hq, Hk, D, R, ty, norm, inter, weights, far, fused)
    r, dt = Rand(seed), TYPES[ty]
    if fused:
        qkv = r(B, T, Hq + 2 * Hk, D, dtype=dt)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        on = qkv.to(DEV)
        gq, gk = on[:, :, :Hq].detach().requires_grad_(True), on[:, :, Hq:Hq + Hk].detach().requires_grad_(True)
    else:
        q, k = r(B, T, Hq, D, dtype=dt), r(B, T, Hk, D, dtype=dt)
        gq, gk = (t.to(DEV).requires_grad_(True) for t in (q, k))
    ws = [1 + r(D, std=0.3) if weights else None for _ in range(2)]
    gw = [None if w is None else w.to(DEV).requires_grad_(True) for w in ws]
    pos = (far + torch.arange(T) * 3 - 2).expand(B, T).contiguous().to(torch.int32)
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)) if R else None
    cq, ck = r(B, T, Hq, D, dtype=dt), r(B, T, Hk, D, dtype=dt)
    outs = kda_qk_norm_rope(gq, gk, dev(pos), dev(f), q_weight=gw[0], k_weight=gw[1], norm=norm, interleaved=inter)
    leaves = [t for t in (gq, gk, *gw) if t is not None]
    got = torch.autograd.grad(outs, leaves, (dev(cq), dev(ck)))
    torch.cuda.synchronize()
    half = HALF[dt]
    # 2^-18: the hardware's sines; else 2^-20: 20 roundings of sums and 12 of products
    e = (2.0 ** -18 if ty == "bf16" else 2.0 ** -20) + 32 * 2.0 ** -24
    count = D if norm == "rms" else 1
    for i, (x, w, c) in enumerate(((q, ws[0], cq), (k, ws[1], ck))):
        fn = lambda x, w: A.qk_norm_rope(x, pos, f, w, norm, interleaved=inter)  # noqa: E731
        (o,), g = A.grads(fn, [x, w], [c])
        # a turned pair is off relative to the pair's size; the largest channel of the row bounds it
        top = lambda t: t.abs().amax(-1, keepdim=True).expand(t.shape) if t.numel() else t  # noqa: E731
        near(f"out{i}", outs[i], o, half * o.abs() + 2 * e * top(o))
        n = A.qk_norm_rope(A.f64(x), None, None, None, norm)
        rr = n.abs().amax(-1, keepdim=True) / A.f64(x).abs().amax(-1, keepdim=True).clamp(min=1e-300)
        dn = 2 * top(A.f64(c)) * (1 if w is None else w.abs().max().item())
        size = rr * (dn + top(n) * (dn * n.abs()).sum(-1, keepdim=True) / count) if norm != "none" else dn
        near(f"dx{i}", got[i], g[0], half * g[0].abs() + 4 * e * size)
        if w is not None:
            terms = (2 * top(A.f64(c)) * n.abs()).sum((0, 1, 2))
            near(f"dw{i}", got[2 + i], g[1], 2.0 ** -24 * g[1].abs() + 4 * e * terms)


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [(1, 1, 1, 1, 8, 8), (2, 5, 3, 1, 64, 64), (1, 33, 7, 2, 80, 32),
                                           (1, 70, 4, 4, 128, 64), (3, 3, 1, 6, 512, 128), (1, 19, 9, 3, 24, 16)])
def test_qk(B, T, Hq, Hk, D, R, inter, norm, ty):
    qk_check(21, B, T, Hq, Hk, D, R, ty, norm, inter, weights=norm != "none" and T != 5, fused=T == 33)


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("far", [1 << 20, 2147480000, -5000000])
def test_qk_at_far_positions(far, ty):
    qk_check(22, 1, 40, 2, 2, 64, 64, ty, far=far)


def test_qk_without_rotation_and_many_rows():
    qk_check(23, 2, 9, 4, 2, 96, 0, norm="rms", weights=True)
    qk_check(24, 1, 700, 24, 8, 128, 128, norm="rms", weights=True, fused=True)  # more items than the backward's grid


def test_qk_zero_rows_empty_calls_and_in_place():
    q = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 1] = 2.0
    k = torch.randn(1, 3, 2, 64, device=DEV).bfloat16()
    pos = torch.tensor([[1, 2, 3]], dtype=torch.int32, device=DEV)
    f = torch.tensor([1.0, 0.1], dtype=torch.float64, device=DEV).repeat(16)
    a, b = kda_qk_norm_rope(q, k, pos, f)
    assert not a[0, 0].any() and not a[0, 2].any() and torch.isfinite(a.float()).all()
    e = kda_qk_norm_rope(q[:, :0], k[:, :0], pos[:, :0], f)
    assert e[0].shape == (1, 0, 2, 64)
    only, none = kda_qk_norm_rope(q, k[:, :, :0], pos, f)
    assert torch.equal(only, a) and none.numel() == 0
    wide = torch.stack([q, k], 2).flatten(2, 3)  # [1, 3, 4, 64]: q and k heads side by side
    vq, vk = wide[:, :, :2], wide[:, :, 2:]
    kda.kda_qk_rope_fwd(vq, vk, vq, vk, pos, f)
    assert torch.equal(vq, a) and torch.equal(vk, b)
    with pytest.raises(ValueError):
        kda.kda_qk_rope_fwd(vq, vk, vq[:, :2], vk, pos, f)
    # rows as large as bf16 goes whose squares still fit fp32, and infinities, stay in their row
    k[0, 0, 0], k[0, 2, 1, 5] = 1e18, float("inf")
    _, c = kda_qk_norm_rope(q, k, pos, f)
    keep = torch.ones(3, 2, dtype=torch.bool)
    keep[0, 0] = keep[2, 1] = False
    assert torch.equal(c[0].cpu()[keep], b[0].cpu()[keep]) and torch.isfinite(c[0, 0, 0].float()).all()


# ---------------------------------------------------------------------------
# together, on other streams, captured
# ---------------------------------------------------------------------------
def test_a_layer_of_them_with_the_core():
    """Convolutions in front of q, k, v and of the recurrence, norm and rotation of q and k, then the
    chunked core on the unit rows (FLAG_NO_QK_NORM): each stage against its oracle on the stage's own
    inputs, and packed sequences against the same sequences alone."""
    import oracle

    H, K, cu = 2, 64, [0, 70, 70, 133, 200]
    r = Rand(31)
    proj = r(1, 200, 3 * H * K, dtype=torch.bfloat16)
    w = [r(H * K, 4, std=0.5) for _ in range(3)]
    g, b = r(1, 200, H, K, dtype=torch.bfloat16), r(1, 200, H, dtype=torch.bfloat16)
    al, dt = r(H, std=0.5), r(H, K, std=0.1)
    pos = torch.cat([torch.arange(hi - lo) for lo, hi in zip(cu[:-1], cu[1:])])[None].to(torch.int32)
    f = 10000.0 ** (-torch.arange(0, K, 2, dtype=torch.float64) / K)

    def layer(lo, hi, cu):
        cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
        at = lambda t: t[:, lo:hi].to(DEV)  # noqa: E731
        p = at(proj)
        with torch.no_grad():
            q, k, v = (kda_short_conv(p[..., i * H * K:(i + 1) * H * K], dev(w[i]), cu_seqlens=cu)[0].view(1, hi - lo, H, K)
                       for i in range(3))
            qn, kn = kda_qk_norm_rope(q, k, at(pos), dev(f))
            out, N = torch.empty_like(v), 1 if cu is None else cu.numel() - 1
            fin = torch.empty(N, H, K, K, device=DEV)
            ws = torch.empty(kda.kda_workspace_size(hi - lo, H, N), dtype=torch.uint8, device=DEV)
            kda.kda_fwd_ex(qn, kn, v, at(g).contiguous(), at(b).contiguous(), K ** -0.5, out, ws, dev(al), dev(dt), -5.0,
                           None, fin, cu, flags=kda.FLAG_NO_QK_NORM)
            rec, rfin = kda_glr(v, at(g).contiguous(), dev(al), dev(dt), cu_seqlens=cu, complement=True)
        torch.cuda.synchronize()
        assert kda.kda_workspace_faults(ws) == 0
        return [t.cpu() for t in (q, k, v, qn, kn, out, fin, rec, rfin)]

    q, k, v, qn, kn, out, fin, rec, rfin = layer(0, 200, cu)
    for i, t in enumerate((q, k, v)):
        x = proj[..., i * H * K:(i + 1) * H * K]
        o, _ = A.conv(A.f64(x), A.f64(w[i]), None, None, cu)
        near("conv", t, o, 2.0 ** -8 * o.abs() + 2.0 ** -18)
    for t, n in ((q, qn), (k, kn)):
        o = A.qk_norm_rope(A.f64(t), pos, f)
        near("rope", n, o, 2.0 ** -8 * o.abs() + 2.0 ** -17)
    ref, rf = oracle.oracle_fwd(qn, kn, v, g, b, K ** -0.5, al, dt, -5.0, None, torch.tensor(cu, dtype=torch.int32),
                                flags=kda.FLAG_NO_QK_NORM)
    m = oracle.metrics(out.double().numpy().reshape(ref.shape), ref)
    assert m["finite"] and m["rel_l2"] <= 1e-2 and m["max_abs"] <= 3e-2
    c = dict(x=v, g=g, al=al, dt=dt, init=None, cu=torch.tensor(cu), given=False, complement=True,
             d_out=torch.zeros_like(v), d_fin=torch.zeros(4, H, K))
    (o, ff), _ = glr_oracle(c, grad=False)
    t = glr_bounds(c)
    near("glr", rec, o, t["out"] + 2.0 ** -8 * o.abs())
    near("glr state", rfin, ff, t["fin"] + 2.0 ** -24 * ff.abs())
    for n in (0, 2, 3):
        lo, hi = cu[n], cu[n + 1]
        alone = layer(lo, hi, None)
        for name, a, whole in zip("q k v qn kn".split(), alone, (q, k, v, qn, kn)):
            assert torch.equal(a, whole[:, lo:hi]), name  # row by row the same arithmetic
        assert torch.allclose(alone[5].float(), out[:, lo:hi].float(), atol=2e-3, rtol=2.0 ** -7)
        assert torch.allclose(alone[7].float(), rec[:, lo:hi].float(), atol=1e-5, rtol=2.0 ** -7)


def test_gradients_through_the_layer():
    """Gradients reach the projection and every parameter through all stages with the core in between."""
    r, H, K, T = Rand(32), 2, 64, 96
    leaf = lambda t: t.to(DEV).requires_grad_(True)  # noqa: E731
    proj = leaf(r(1, T, 3 * H * K, dtype=torch.bfloat16))
    w = [leaf(r(H * K, 4, std=0.5)) for _ in range(3)]
    wq, wk = leaf(1 + r(K, std=0.1)), leaf(1 + r(K, std=0.1))
    al, dt = leaf(r(H, std=0.5)), leaf(r(H, K, std=0.1))
    g, b = leaf(r(1, T, H, K, dtype=torch.bfloat16)), leaf(r(1, T, H, dtype=torch.bfloat16))
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV)[None], torch.ones(16, dtype=torch.float64, device=DEV)
    q, k, v = (kda_short_conv(proj[..., i * H * K:(i + 1) * H * K], w[i])[0].view(1, T, H, K) for i in range(3))
    q, k = kda_qk_norm_rope(q, k, pos, f, q_weight=wq, k_weight=wk)
    out, _ = kda_chunk(q, k, v, g, b, al, dt)
    rec, _ = kda_glr(out, g, al, dt, complement=True)
    leaves = [proj, *w, wq, wk, al, dt, g, b]
    grads = torch.autograd.grad((rec.float() * r(1, T, H, K).to(DEV)).sum(), leaves)
    for t, d in zip(leaves, grads):
        assert d.shape == t.shape and torch.isfinite(d).all() and d.abs().max() > 0


def calls(seed):
    """One inference call of each, on preallocated buffers; returns (call, inputs, outputs)."""
    c = glr_case(seed, 1, 0, 3, 64, [200, 0, 333, 67])
    v = conv_case(seed, 1, 0, 192, 4, [200, 0, 333, 67])
    r = Rand(seed)
    d = {("g", k): dev(t) for k, t in c.items() if torch.is_tensor(t)}
    d |= {("c", k): dev(t) for k, t in v.items() if torch.is_tensor(t)}
    d[("q", "q")], d[("q", "k")] = dev(r(1, 600, 3, 64, dtype=torch.bfloat16)), dev(r(1, 600, 2, 64, dtype=torch.bfloat16))
    d[("q", "pos")] = torch.arange(600, dtype=torch.int32, device=DEV)[None] + seed
    d[("q", "f")] = torch.rand(16, dtype=torch.float64).to(DEV) if seed < 0 else torch.full((16,), 0.3, dtype=torch.float64, device=DEV)
    x, y = d[("g", "x")], d[("c", "x")]
    o = dict(out=torch.empty_like(x), fin=torch.empty(4, 3, 64, device=DEV), dx=torch.empty_like(x), dg=torch.empty_like(x),
             dA=torch.empty(3, device=DEV), dd=torch.empty(3, 64, device=DEV), di=torch.empty(4, 3, 64, device=DEV),
             y=torch.empty_like(y), cf=torch.empty(4, 3, 192, device=DEV, dtype=y.dtype), dy=torch.empty_like(y),
             dw=torch.empty(192, 4, device=DEV), db=torch.empty(192, device=DEV),
             qo=torch.empty_like(d[("q", "q")]), ko=torch.empty_like(d[("q", "k")]),
             dq=torch.empty_like(d[("q", "q")]), dk=torch.empty_like(d[("q", "k")]), dqw=torch.empty(64, device=DEV))
    size = max(kda.kda_glr_bwd_workspace_size(600, 3, 64), kda.kda_conv_bwd_workspace_size(600, 192, 4),
               kda.kda_qk_rope_bwd_workspace_size(600, 3, 2, 64))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    st = torch.empty(kda.kda_glr_states_size(600, 3, 64), dtype=torch.uint8, device=DEV)
    G = lambda n: d[("g", n)]  # noqa: E731
    C = lambda n: d[("c", n)]  # noqa: E731
    Q = lambda n: d[("q", n)]  # noqa: E731

    def call():  # one workspace serves them all, one after the other
        kda.kda_glr_fwd(G("x"), G("g"), o["out"], ws, G("al"), G("dt"), -5.0, G("init"), o["fin"], st, G("cu"))
        kda.kda_glr_bwd(G("x"), G("g"), st, G("d_out"), o["dx"], o["dg"], o["dA"], o["dd"], ws, G("al"), G("dt"), -5.0,
                        G("init"), G("d_fin"), o["di"], G("cu"))
        kda.kda_conv_fwd(C("x"), C("w"), o["y"], C("b"), C("init"), o["cf"], C("cu"), kda.FLAG_SILU)
        kda.kda_conv_bwd(C("x"), C("w"), C("d_out"), o["dy"], o["dw"], ws, C("b"), o["db"], C("init"), C("d_fin"), None,
                         C("cu"), kda.FLAG_SILU)
        kda.kda_qk_rope_fwd(Q("q"), Q("k"), o["qo"], o["ko"], Q("pos"), Q("f"))
        kda.kda_qk_rope_bwd(Q("q"), Q("k"), o["qo"], o["ko"], o["dq"], o["dk"], Q("pos"), Q("f"), d_q_weight=o["dqw"],
                            workspace=ws)

    return call, d, o


def test_captured_and_replayed():
    """All of them in one captured graph, both directions; replays with new inputs, eager work between
    them, and the sequences cut elsewhere (cu_seqlens is data)."""
    call, d, o = calls(40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        call()
    torch.cuda.synchronize()
    for i in range(4):
        eager, de, oe = calls(41 + i)
        if i == 2:
            for s in ("g", "c"):
                de[(s, "cu")].copy_(torch.tensor([0, 1, 300, 555, 600], dtype=torch.int32))
        for n in d:
            d[n].copy_(de[n])
        say("replay", i)
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n], oe[n]), (i, n)


def test_two_streams_at_once():
    """Two independent sets of calls, each with its own workspace, on two streams that overlap."""
    a, b = calls(50), calls(51)
    a[0](), b[0]()
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in s[2].items()} for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, st in zip((a, b), streams):
            for t in s[2].values():
                t.zero_()
        torch.cuda.synchronize()
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s[0]()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            assert all(torch.equal(t, w[n]) for n, t in s[2].items())


@pytest.mark.parametrize("cu", [[0, -5, 40], [0, 30, 10, 40], [0, 12, 100], [7, 20, 40], [0, -1, -2], [40, 0, 0]])
def test_offsets_that_break_the_contract_stay_inside(cu):
    """Their results are not specified, but rows in front of and behind the arrays are neither used nor written."""
    T, C, W, pad, r = 40, 64, 4, 8, Rand(60)
    N = len(cu) - 1

    def framed(t, fill=float("nan")):
        whole = torch.full((t.shape[0] + 2 * pad, *t.shape[1:]), fill, dtype=t.dtype, device=DEV)
        whole[pad:-pad] = t.to(DEV)
        return whole, whole[pad:-pad]

    x, g, d_out = (framed(r(T, C, dtype=torch.bfloat16))[1] for _ in range(3))
    outs = {n: framed(torch.zeros(T, C, dtype=torch.bfloat16), 7.0) for n in ("h", "dx", "dg", "y", "dy")}
    states = {n: framed(torch.zeros(N, C), 7.0) for n in ("fin", "di")}
    rows = {n: framed(torch.zeros(N, W - 1, C, dtype=torch.bfloat16), 7.0) for n in ("cf", "cd")}
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    al, dt, w, init = dev(r(1)), dev(r(1, C)), dev(r(C, W)), dev(r(N, W - 1, C, dtype=torch.bfloat16))
    four, o = lambda t: t.view(1, T, 1, C), lambda n: outs[n][1]  # noqa: E731
    ws = torch.empty(max(kda.kda_glr_bwd_workspace_size(T, 1, C), kda.kda_conv_bwd_workspace_size(T, C, W)),
                     dtype=torch.uint8, device=DEV)
    kept = torch.empty(kda.kda_glr_states_size(T, 1, C), dtype=torch.uint8, device=DEV)
    dA, dd, dw = torch.empty(1, device=DEV), torch.empty(1, C, device=DEV), torch.empty(C, W, device=DEV)
    say("glr", cu.tolist())
    kda.kda_glr_fwd(four(x), four(g), four(o("h")), ws, al, dt, -5.0, None, states["fin"][1].view(N, 1, C), kept, cu)
    torch.cuda.synchronize()
    assert kda.kda_workspace_faults(ws) == 0
    kda.kda_glr_bwd(four(x), four(g), kept, four(d_out), four(o("dx")), four(o("dg")), dA, dd, ws, al, dt, -5.0, None, None,
                    states["di"][1].view(N, 1, C), cu)
    torch.cuda.synchronize()
    assert kda.kda_workspace_faults(ws) == 0
    say("conv", cu.tolist())
    kda.kda_conv_fwd(x[None], w, o("y")[None], None, init, rows["cf"][1], cu, kda.FLAG_SILU)
    kda.kda_conv_bwd(x[None], w, d_out[None], o("dy")[None], dw, ws, None, None, init, None, rows["cd"][1], cu, kda.FLAG_SILU)
    torch.cuda.synchronize()
    for n, (whole, inner) in (outs | states | rows).items():
        assert torch.isfinite(inner).all(), n
        assert (whole[:pad] == 7).all() and (whole[-pad:] == 7).all(), n
    assert all(torch.isfinite(t).all() for t in (dA, dd, dw))


def test_captured_training_pass():
    """Forward and backward through autograd in one captured graph, replayed with new inputs; the eager
    passes between the replays have leaves of their own."""
    H, K, T = 2, 64, 300
    cu = torch.tensor([0, 120, 120, 290], dtype=torch.int32, device=DEV)
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV)[None], torch.full((16,), 0.3, dtype=torch.float64, device=DEV)

    def inputs(seed):
        r = Rand(seed)
        leaves = [r(1, T, H * K, dtype=torch.bfloat16), r(H * K, 4, std=0.5), r(H * K), 1 + r(K, std=0.1), r(1, T, H, K, dtype=torch.bfloat16),
                  r(H, std=0.5), r(H, K, std=0.1), r(3, H, K)]
        return [t.to(DEV).requires_grad_(True) for t in leaves], [dev(r(1, T, H, K, dtype=torch.bfloat16)), dev(r(3, H, K))]

    def step(leaves, d):
        x, w, b, nw, g, al, dt, init = leaves
        y = kda_short_conv(x, w, b, cu_seqlens=cu)[0].view(1, T, H, K)
        y, z = kda_qk_norm_rope(y, y, pos, f, q_weight=nw)
        h, fin = kda_glr(y, g, al, dt, initial_state=init, cu_seqlens=cu, complement=True)
        h2, _ = kda_glr(z, g, al, dt, cu_seqlens=cu)
        return torch.autograd.grad((h, fin, h2), leaves, (d[0], d[1], d[0]))

    leaves, d = inputs(70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(leaves, d)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        grads = step(leaves, d)
    torch.cuda.synchronize()
    for i in range(4):
        eager, de = inputs(71 + i)
        with torch.no_grad():
            for to, by in zip(leaves + d, eager + de):
                to.copy_(by)
        say("replay", i)
        graph.replay()
        want = step(eager, de)
        torch.cuda.synchronize()
        for n, (got, w) in enumerate(zip(grads, want)):
            assert torch.equal(got, w), (i, n)
