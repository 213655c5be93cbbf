"""Cases and plain forms of the operators around the KDA core: the gated linear recurrence,
the short causal convolution, and the per-head norm and rotation of queries and keys.

``run(prepare(case, seed))`` is one pass of one operator.  With ``own`` false it is computed
by elementary torch operations in 32 bits (64 for the angles of far positions and for sums
over tokens), rounded once at the end; with ``own`` true by the calls that a user of
``chunked_gated_delta_amd`` makes.  ``exact`` gives the same outputs from the definitions in
64 bits.

Layouts are the library's: per-token tensors [B, T, H, K] (the convolution: [B, T, C]), fp32
parameters, fp32 recurrent states [N, H, K], and packed batches as int32 offsets
``cu_seqlens`` [N + 1] with B = 1.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LOWER_BOUND = -5.0
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _glr(name, mode, B, T, H, K, seqs=0, init=False, complement=False, given=False, type="bf16"):
    return dict(name=name, op="glr", mode=mode, B=B, T=T, H=H, K=K, seqs=seqs, init=init, complement=complement,
                given=given, type=type)


def _conv(name, mode, B, T, C, W=4, seqs=0, init=False, silu=True, bias=False, type="bf16"):
    return dict(name=name, op="conv", mode=mode, B=B, T=T, C=C, W=W, seqs=seqs, init=init, silu=silu, bias=bias,
                type=type)


def _qk(name, mode, B, T, Hq, Hk, D, R, norm="l2", weights=False, interleaved=False, fused=False, far=0,
        type="bf16"):
    return dict(name=name, op="qk", mode=mode, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, norm=norm, weights=weights,
                interleaved=interleaved, fused=fused, far=far, type=type)


def listed():
    return [
        # one 200-token prompt of a two-head layer: the library's smallest shape, launch latency
        _glr("glr_short_prompt", "fwd", 1, 200, 2, 128),
        # one token for each of 64 running sequences of a 96-head layer: decoding
        _glr("glr_token", "step", 64, 1, 96, 128, init=True),
        # a long prompt of a 96-head layer: the library's headline shape
        _glr("glr_prompt", "fwd", 1, 32768, 96, 128),
        # one very long sequence on few heads, input scaled by 1 - decay
        _glr("glr_long", "fwd", 1, 262144, 8, 128, init=True, complement=True),
        # a packed training batch of 16 ragged documents with carried states
        _glr("glr_train_packed", "train", 1, 69141, 32, 128, seqs=16, init=True),
        # a training batch in full precision
        _glr("glr_train_fp32", "train", 2, 4096, 12, 64, complement=True, type="fp32"),
        # the convolution in front of q, k or v: the long prompt, the packed batch, one token
        _conv("conv_prompt", "fwd", 1, 32768, 12288),
        _conv("conv_train_packed", "train", 1, 69141, 4096, seqs=16, init=True, bias=True),
        _conv("conv_token", "step", 64, 1, 12288, init=True),
        # queries and keys of the long prompt, L2 norm and half of the channels rotated
        _qk("qk_prompt", "fwd", 1, 32768, 96, 96, 128, 64),
        # a training batch with 32 query and 8 key heads, taken out of one projection's output
        _qk("qk_train_shared_heads", "train", 2, 4097, 32, 8, 128, 128, norm="rms", weights=True, fused=True),
        # one token for each of 64 sequences at far positions
        _qk("qk_token", "fwd", 64, 1, 96, 96, 128, 64, far=1 << 20),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr", "glr", "conv", "qk"])
    mode = rng.choice(["fwd", "train", "step"]) if op != "qk" else rng.choice(["fwd", "train"])
    type = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    most = 1 << 26  # elements of one tensor
    if op == "qk":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        R = rng.choice([D // 16 * 16, D // 32 * 16, 0])
        Hq = _log(rng, 1, 96)
        Hk = rng.choice([Hq, max(1, Hq // 8), _log(rng, 1, 16)])
        T = _log(rng, 1, max(1, min(65536, most // ((Hq + Hk) * D))))
        B = rng.choice([1, 1, 2, 3])
        norm = rng.choice(["l2", "rms", "none"]) if R else rng.choice(["l2", "rms"])
        return _qk("", mode, B, max(1, T // B), Hq, Hk, D, R, norm=norm, weights=norm != "none" and rng.random() < 0.5,
                   interleaved=rng.random() < 0.3, fused=rng.random() < 0.5, far=rng.choice([0, 0, 1 << 20]),
                   type=type)
    H, K = _log(rng, 1, 96), rng.choice([32, 64, 96, 128, 128, 256])
    if mode == "step":
        B, T, seqs = _log(rng, 1, 512), rng.choice([1, 1, 1, 2, 4]), 0
    else:
        T = _log(rng, 1, min(262144, most // (H * K)))
        B = rng.choice([1, 1, 2, 5])
        T = max(1, T // B)
        seqs = _log(rng, 2, 64) if B == 1 and rng.random() < 0.5 else 0
    init = mode == "step" or rng.random() < 0.5
    if op == "glr":
        return _glr("", mode, B, T, H, K, seqs=seqs, init=init, complement=rng.random() < 0.4,
                    given=rng.random() < 0.25, type=type)
    return _conv("", mode, B, T, H * K, W=rng.choice([2, 3, 4, 4]), seqs=seqs, init=init, silu=rng.random() < 0.7,
                 bias=rng.random() < 0.5, type=type)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ty = TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo, hi):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = dict(case)
    B, T = case["B"], case["T"]
    if case["op"] == "qk":
        Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
        if case["fused"]:  # views of one projection's output, values behind the keys
            qkv = normal(B, T, Hq + 2 * Hk, D, dtype=ty)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = normal(B, T, Hq, D, dtype=ty), normal(B, T, Hk, D, dtype=ty)
        s["q_weight"] = 1.0 + normal(D, std=0.2) if case["weights"] else None
        s["k_weight"] = 1.0 + normal(D, std=0.2) if case["weights"] else None
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / max(R, 1))
        if case["mode"] == "train":
            s["d_q"], s["d_k"] = normal(B, T, Hq, D, dtype=ty), normal(B, T, Hk, D, dtype=ty)
        return s
    n = case["seqs"] or B
    s["cu_seqlens"] = None
    if case["seqs"]:  # ragged documents between sorted cuts: short and empty ones among them
        cuts = torch.randint(0, T + 1, (n - 1,), generator=gen, device=dev).sort().values
        ends = torch.tensor([0, T], device=dev)
        s["cu_seqlens"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    if case["op"] == "glr":
        H, K = case["H"], case["K"]
        s["x"] = normal(B, T, H, K, dtype=ty)
        s["A_log"], s["dt_bias"] = uniform(H, lo=0.0, hi=math.log(16.0)), normal(H, K, std=0.1)
        raw = normal(B, T, H, K)
        if case["given"]:  # the log-decay itself, between the bound and zero
            raw = LOWER_BOUND * torch.sigmoid(raw * 2.0)
            s["A_log"] = s["dt_bias"] = None
        s["raw_gate"] = raw.to(ty)
        s["initial_state"] = normal(n, H, K, std=0.5) if case["init"] else None
        if case["mode"] == "train":
            s["d_out"], s["d_final"] = normal(B, T, H, K, dtype=ty), normal(n, H, K)
    else:
        C, W = case["C"], case["W"]
        s["x"] = normal(B, T, C, dtype=ty)
        s["weight"], s["bias"] = normal(C, W, std=W ** -0.5), normal(C, std=0.1) if case["bias"] else None
        s["initial_state"] = normal(n, W - 1, C, dtype=ty) if case["init"] else None
        if case["mode"] == "train":
            s["d_out"], s["d_final"] = normal(B, T, C, dtype=ty), normal(n, W - 1, C, dtype=ty)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _bounds(s):
    """First token and length of each sequence on the packed axis [B * T]."""
    if s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].long()
        return cu[:-1], cu[1:] - cu[:-1]
    first = torch.arange(s["B"], device=s["x"].device) * s["T"]
    return first, torch.full_like(first, s["T"])


def _most(s):
    """An upper bound of the longest sequence that needs no look at device data."""
    return s["T"]


def _glr_gate(s):
    """z, sigma(z) (None where the decay is given) and the log-decay g, fp32 [B * T, H, K]."""
    raw = s["raw_gate"].float().flatten(0, 1)
    if s["given"]:
        return None, None, raw
    z = torch.exp(s["A_log"])[:, None] * (raw + s["dt_bias"])
    sig = torch.sigmoid(z)
    return z, sig, LOWER_BOUND * sig


def _edges(first, length, M):
    """Where sequences with tokens start and end: the token's row, its sequence; and rows of M."""
    n = torch.arange(first.numel(), device=first.device)
    has = length > 0
    at_first = torch.full((M,), -1, device=first.device, dtype=torch.long)
    at_last = at_first.clone()
    spare = torch.where(has, first, M)  # empty sequences go to a row that is cut off
    at_first = torch.cat([at_first, at_first[:1]]).index_copy_(0, spare, n)[:M] if M else at_first
    spare = torch.where(has, first + length - 1, M)
    at_last = torch.cat([at_last, at_last[:1]]).index_copy_(0, spare, n)[:M] if M else at_last
    return at_first, at_last


def _scan(a, u, most):
    """u_t + a_t h_{t-1} for all t by doubling: after the step of distance d every row holds the
    map of its last 2 d tokens.  The rows where a sequence starts have a = 0."""
    d = 1
    while d < min(most, u.shape[0]):
        u[d:] = u[d:] + a[d:] * u[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return u


def _plain_glr(s):
    x = s["x"].float().flatten(0, 1)
    M = x.shape[0]
    first, length = _bounds(s)
    at_first, at_last = _edges(first, length, M)
    z, sig, g = _glr_gate(s)
    a = torch.exp(g)
    b = -torch.expm1(g) if s["complement"] else None
    u = x if b is None else b * x
    start = (at_first >= 0)[:, None, None]
    N = first.numel()
    init = s["initial_state"]
    if init is None:
        init = torch.zeros(N, *x.shape[1:], device=x.device)
    enter = init[at_first.clamp(min=0)] * start  # the state that a sequence's first token meets
    h = _scan(torch.where(start, 0.0, a), u + a * enter, _most(s))
    last = (first + length - 1).clamp(min=0)
    final = torch.where((length > 0)[:, None, None], h[last], init)
    out = h.to(s["x"].dtype).view_as(s["x"])
    if s["mode"] != "train":
        return out, final
    # backward: dh_t = d_out_t + a_{t+1} dh_{t+1}, the last token also gets d_final
    end = (at_last >= 0)[:, None, None]
    dh = s["d_out"].float().flatten(0, 1) + s["d_final"][at_last.clamp(min=0)] * end
    nxt = torch.where(end, 0.0, torch.cat([a[1:], a[:1]]))
    dh = _scan(nxt.flip(0), dh.flip(0), _most(s)).flip(0)
    before = torch.where(start, enter, torch.cat([h[:1], h[:-1]]))
    dx = dh if b is None else dh * b
    da = dh * before if b is None else dh * (before - x)
    dg = da * a
    d_init = torch.where((length > 0)[:, None, None], (a * dh)[first.clamp(max=M - 1)], s["d_final"])
    grads = [dx.to(s["x"].dtype).view_as(s["x"])]
    if s["given"]:
        grads += [dg.to(s["x"].dtype).view_as(s["x"])]
    else:
        dz = dg * (LOWER_BOUND * sig * (1.0 - sig))
        draw = dz * torch.exp(s["A_log"])[:, None]
        grads += [draw.to(s["x"].dtype).view_as(s["x"]), (dz * z).sum((0, 2), dtype=torch.float64).float(),
                  draw.sum(0, dtype=torch.float64).float()]
    return (out, final, *grads, *([d_init] if s["init"] else []))


def _conv_rows(s):
    """The inputs that token t's taps meet, as rows of [x; state rows]: index [B * T, W]."""
    first, length = _bounds(s)
    W, M = s["W"], s["B"] * s["T"]
    t = torch.arange(M, device=first.device)
    n = torch.searchsorted((first + length), t, right=True)
    back = t[:, None] - first[n][:, None] + torch.arange(W, device=t.device) - (W - 1)  # within the sequence
    row = torch.where(back >= 0, first[n][:, None] + back, M + n[:, None] * (W - 1) + back + W - 1)
    # the state that is left: the last W - 1 inputs, older state rows where the sequence is short
    keep = length[:, None] + torch.arange(W - 1, device=t.device) - (W - 1)
    seq = torch.arange(first.numel(), device=t.device)[:, None]
    left = torch.where(keep >= 0, first[:, None] + keep, M + seq * (W - 1) + keep + W - 1)
    return row, left


def _plain_conv(s):
    ty, W, C = s["x"].dtype, s["W"], s["C"]
    M, N = s["B"] * s["T"], s["seqs"] or s["B"]
    init = s["initial_state"]
    if init is None:
        init = torch.zeros(N, W - 1, C, device=s["x"].device)
    ext = torch.cat([s["x"].reshape(M, C), init.to(ty).reshape(-1, C)]).float()
    row, left = _conv_rows(s)
    z = sum(s["weight"][:, j] * ext[row[:, j]] for j in range(W))
    z = z if s["bias"] is None else z + s["bias"]
    y = z * torch.sigmoid(z) if s["silu"] else z
    out, final = y.to(ty).view_as(s["x"]), ext[left].to(ty)
    if s["mode"] != "train":
        return out, final
    dz = s["d_out"].float().reshape(M, C)
    if s["silu"]:
        sig = torch.sigmoid(z)
        dz = dz * (sig * (1.0 + z * (1.0 - sig)))
    d = torch.zeros_like(ext)
    [d.index_add_(0, row[:, j], dz * s["weight"][:, j]) for j in range(W)]
    d.index_add_(0, left.flatten(), s["d_final"].float().reshape(-1, C))
    dw = torch.stack([(dz * ext[row[:, j]]).sum(0, dtype=torch.float64).float() for j in range(W)], 1)
    grads = [d[:M].to(ty).view_as(s["x"]), dw]
    grads += [] if s["bias"] is None else [dz.sum(0, dtype=torch.float64).float()]
    grads += [d[M:].to(ty).view(N, W - 1, C)] if s["init"] else []
    return (out, final, *grads)


def _turn(x, cos, sin, R, interleaved):
    if R == 0:
        return x
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_qk(s):
    R, inter = s["R"], s["interleaved"]
    angle = s["positions"].double()[..., None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    outs, grads = [], []
    parts = [(s["q"], s["q_weight"], "d_q"), (s["k"], s["k_weight"], "d_k")]

    def one(x, w, dy):
        f = x.float()
        count = f.shape[-1] if s["norm"] == "rms" else 1
        r = torch.rsqrt((f * f).sum(-1, keepdim=True) / count + EPS) if s["norm"] != "none" else None
        n = f if r is None else f * r
        outs.append(_turn(n if w is None else n * w, cos, sin, R, inter).to(x.dtype))
        if s["mode"] == "train":
            dn = _turn(s[dy].float(), cos, -sin, R, inter)
            dw = None if w is None else (dn * n).sum((0, 1, 2), dtype=torch.float64).float()
            dn = dn if w is None else dn * w
            dx = dn if r is None else r * (dn - n * ((dn * n).sum(-1, keepdim=True) / count))
            grads.append((dx.to(x.dtype), dw))

    [one(*p) for p in parts]
    return (*outs, *(t for g in grads for t in g if t is not None))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_glr(s):
    import chunked_gated_delta_amd as kda
    from chunked_gated_delta_amd.function import kda_glr

    x, raw, al, dt, init = s["x"], s["raw_gate"], s["A_log"], s["dt_bias"], s["initial_state"]
    if s["mode"] == "step":
        out, final = torch.empty_like(x), torch.empty_like(init)
        flags = (kda.FLAG_GATE_GIVEN if s["given"] else 0) | (kda.FLAG_COMPLEMENT if s["complement"] else 0)
        kda.kda_glr_step(x, raw, out, al, dt, LOWER_BOUND, initial_state=init, final_state=final, flags=flags)
        return out, final
    kw = dict(lower_bound=LOWER_BOUND, cu_seqlens=s["cu_seqlens"], gate_given=s["given"], complement=s["complement"])
    if s["mode"] == "fwd":
        return kda_glr(x, raw, al, dt, initial_state=init, **kw)
    leaves = [t.detach().requires_grad_() for t in (x, raw, al, dt, init) if t is not None]
    it = iter(leaves)
    x, raw, al, dt, init = (None if t is None else next(it) for t in (x, raw, al, dt, init))
    out, final = kda_glr(x, raw, al, dt, initial_state=init, **kw)
    return (out, final, *torch.autograd.grad((out, final), leaves, (s["d_out"], s["d_final"])))


def _own_conv(s):
    import chunked_gated_delta_amd as kda
    from chunked_gated_delta_amd.function import kda_short_conv

    x, w, b, init = s["x"], s["weight"], s["bias"], s["initial_state"]
    if s["mode"] == "step":
        out, final = torch.empty_like(x), torch.empty_like(init)
        kda.kda_conv_step(x, w, out, bias=b, initial_state=init, final_state=final,
                          flags=kda.FLAG_SILU if s["silu"] else 0)
        return out, final
    kw = dict(silu=s["silu"], cu_seqlens=s["cu_seqlens"])
    if s["mode"] == "fwd":
        return kda_short_conv(x, w, b, initial_state=init, **kw)
    leaves = [t.detach().requires_grad_() for t in (x, w, b, init) if t is not None]
    it = iter(leaves)
    x, w, b, init = (None if t is None else next(it) for t in (x, w, b, init))
    out, final = kda_short_conv(x, w, b, initial_state=init, **kw)
    return (out, final, *torch.autograd.grad((out, final), leaves, (s["d_out"], s["d_final"])))


def _own_qk(s):
    from chunked_gated_delta_amd.function import kda_qk_norm_rope

    kw = dict(norm=s["norm"], eps=EPS, interleaved=s["interleaved"])
    q, k, qw, kw_ = s["q"], s["k"], s["q_weight"], s["k_weight"]
    if s["mode"] == "fwd":
        return kda_qk_norm_rope(q, k, s["positions"], s["inv_freq"], q_weight=qw, k_weight=kw_, **kw)
    leaves = [t.detach().requires_grad_() for t in (q, qw, k, kw_) if t is not None]
    it = iter(leaves)
    q, qw, k, kw_ = (None if t is None else next(it) for t in (q, qw, k, kw_))
    outs = kda_qk_norm_rope(q, k, s["positions"], s["inv_freq"], q_weight=qw, k_weight=kw_, **kw)
    return (*outs, *torch.autograd.grad(outs, leaves, (s["d_q"], s["d_k"])))


def run(state):
    op = state["op"]
    if own:
        return {"glr": _own_glr, "conv": _own_conv, "qk": _own_qk}[op](state)
    return {"glr": _plain_glr, "conv": _plain_conv, "qk": _plain_qk}[op](state)


def work(case):
    """Each input read once, each output written once; operations of the formulas."""
    es, M, train = (2 if case["type"] == "bf16" else 4), case["B"] * case["T"], case["mode"] == "train"
    if case["op"] == "qk":
        R, D, heads = case["R"], case["D"], case["Hq"] + case["Hk"]
        elements = M * heads * D
        wide = 2 * D * 4 if case["weights"] else 0
        return {"bytes": elements * es * (4 if train else 2) + M * 4 + R * 4 + wide * (2 if train else 1),
                "flops": M * heads * ((4 * D + 3 * R) * (3 if train else 1))}
    n = case["seqs"] or case["B"]
    if case["op"] == "glr":
        C = case["H"] * case["K"]
        params = 0 if case["given"] else 4 * (C + case["H"])
        states = n * C * 4 * ((2 if train else 1) * (2 if case["init"] else 1))
        return {"bytes": M * C * es * (6 if train else 3) + params * (2 if train else 1) + states,
                "flops": M * C * (30 if train else 12)}
    C, W = case["C"], case["W"]
    states = n * (W - 1) * C * es * ((2 if train else 1) * (2 if case["init"] else 1))
    params = 4 * C * (W + (1 if case["bias"] else 0))
    return {"bytes": M * C * es * (4 if train else 2) + params * (2 if train else 1) + states,
            "flops": M * C * (2 * W + 4) * (3 if train else 1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _sequences(s):
    cu = [b * s["T"] for b in range(s["B"] + 1)] if s["cu_seqlens"] is None else s["cu_seqlens"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_glr(s):
    """Token by token, as the recurrence is written; the gradients token by token backwards."""
    H, K = s["H"], s["K"]
    x, raw = (s[n].double().reshape(-1, H, K) for n in ("x", "raw_gate"))
    if s["given"]:
        g = raw
    else:
        z = s["A_log"].double().exp()[:, None] * (raw + s["dt_bias"].double())
        sig = 1.0 / (1.0 + torch.exp(-z))
        g = LOWER_BOUND * sig
    a = g.exp()
    b = -torch.expm1(g) if s["complement"] else torch.ones_like(g)
    u = b * x
    seqs = _sequences(s)
    init = torch.zeros(len(seqs), H, K, dtype=torch.float64, device=x.device) if s["initial_state"] is None \
        else s["initial_state"].double()
    h, before, final = torch.empty_like(x), torch.empty_like(x), init.clone()
    for n, (lo, hi) in enumerate(seqs):
        state = init[n]
        for t in range(lo, hi):
            state = torch.addcmul(u[t], a[t], state, out=h[t])
        if hi > lo:
            before[lo], before[lo + 1:hi], final[n] = init[n], h[lo:hi - 1], h[hi - 1]
    if s["mode"] != "train":
        return h.view(s["x"].shape), final
    d_out = s["d_out"].double().reshape(-1, H, K)
    dh, d_init = torch.empty_like(x), s["d_final"].double().clone()
    for n, (lo, hi) in enumerate(seqs):
        down = s["d_final"][n].double()
        for t in range(hi - 1, lo - 1, -1):
            torch.add(d_out[t], down, out=dh[t])
            down = a[t] * dh[t]
        d_init[n] = down
    dg = dh * a * (before - x if s["complement"] else before)
    grads = [(dh * b).view(s["x"].shape)]
    if s["given"]:
        grads.append(dg.view(s["x"].shape))
    else:
        dz = dg * LOWER_BOUND * sig * (1.0 - sig)
        draw = dz * s["A_log"].double().exp()[:, None]
        grads += [draw.view(s["x"].shape), (dz * z).sum((0, 2)), draw.sum(0)]
    return (h.view(s["x"].shape), final, *grads, *([d_init] if s["init"] else []))


def _exact_conv(s):
    """Each sequence by itself: its inputs behind its state, taps as shifted products."""
    C, W, train = s["C"], s["W"], s["mode"] == "train"
    leaf = lambda t: None if t is None else t.double().detach().requires_grad_(train)  # noqa: E731
    x, w, bias, init = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"]), leaf(s["initial_state"])
    rows, outs, finals = x.reshape(-1, C), [], []
    for n, (lo, hi) in enumerate(_sequences(s)):
        head = torch.zeros(W - 1, C, dtype=torch.float64, device=x.device) if init is None else init[n]
        line = torch.cat([head, rows[lo:hi]])
        y = torch.zeros(hi - lo, C, dtype=torch.float64, device=x.device) if bias is None else bias.expand(hi - lo, C)
        for j in range(W):
            y = y + line[j:j + hi - lo] * w[:, j]
        outs.append(y / (1.0 + torch.exp(-y)) if s["silu"] else y)
        finals.append(line[hi - lo:])
    out, final = torch.cat(outs).view(s["x"].shape), torch.stack(finals)
    if not train:
        return out, final
    leaves = [t for t in (x, w, bias, init) if t is not None]
    grads = torch.autograd.grad((out, final), leaves, (s["d_out"].double(), s["d_final"].double()))
    return (out.detach(), final.detach(), *grads)


def _exact_qk(s):
    """The rotation as a product with exp(i angle) of complex pairs."""
    R, D, train = s["R"], s["D"], s["mode"] == "train"
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    unit = torch.polar(torch.ones_like(angle), angle)
    outs, grads = [], []
    for x, w, dy in ((s["q"], s["q_weight"], "d_q"), (s["k"], s["k_weight"], "d_k")):
        x = x.double().detach().requires_grad_(train)
        w = None if w is None else w.double().detach().requires_grad_(train)
        y = x
        if s["norm"] != "none":
            y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / (D if s["norm"] == "rms" else 1) + EPS)
        y = y if w is None else y * w
        if R:
            head = y[..., :R]
            re, im = (head[..., 0::2], head[..., 1::2]) if s["interleaved"] else head.split(R // 2, -1)
            pair = torch.complex(re.contiguous(), im.contiguous()) * unit
            head = torch.stack([pair.real, pair.imag], -1).flatten(-2) if s["interleaved"] \
                else torch.cat([pair.real, pair.imag], -1)
            y = torch.cat([head, y[..., R:]], -1)
        outs.append(y.detach())
        if train:
            grads += torch.autograd.grad(y, [t for t in (x, w) if t is not None], s[dy].double())
    return (*outs, *grads)


def exact(case, seed):
    s = prepare(case, seed)
    return {"glr": _exact_glr, "conv": _exact_conv, "qk": _exact_qk}[case["op"]](s)
