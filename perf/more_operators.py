"""Cases and plain forms of the two token mixers that stand beside KDA layers: linear attention
with one decay for each head, and causal attention with grouped heads.

``run(prepare(case, seed))`` is one pass of one operator.  With ``own`` false it is computed by
elementary torch operations in 32 bits and rounded once at the end; with ``own`` true by the
calls that a user of ``chunked_gated_delta_amd`` makes.  ``exact`` gives the same outputs from
the definitions in 64 bits.

Layouts are the library's: token arrays bf16 [B, T, H, K], fp32 states [N, H, K, V], log-sums
fp32 [B, T, H], and packed batches as int32 offsets ``cu_seqlens`` [N + 1] with B = 1.
"""

import math

import torch

own = False

BF16 = torch.bfloat16
CHUNK = 64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _la(name, mode, B, T, H, K=128, V=128, seqs=0, init=False, fused=False):
    return dict(name=name, op="la", mode=mode, B=B, T=T, H=H, K=K, V=V, seqs=seqs, init=init, fused=fused)


def _attn(name, mode, B, T, Hq, Hk, D=128, seqs=0, past=0, fused=False):
    return dict(name=name, op="attn", mode=mode, B=B, T=T, Hq=Hq, Hk=Hk, D=D, seqs=seqs, past=past, fused=fused)


def listed():
    return [
        # one 200-token prompt of a two-head layer: the library's smallest shape, launch latency
        _la("la_short_prompt", "fwd", 1, 200, 2),
        # one token for each of 64 running sequences of a 96-head layer: decoding
        _la("la_token", "step", 64, 1, 96, init=True),
        # a long prompt of a 96-head layer: the library's headline shape
        _la("la_prompt", "fwd", 1, 32768, 96),
        # one very long sequence on few heads, going on from a carried state
        _la("la_long", "fwd", 1, 262144, 8, init=True),
        # a packed training batch of 16 ragged documents with carried states
        _la("la_train_packed", "train", 1, 69141, 32, seqs=16, init=True),
        # one of eight GPUs' share of a training batch
        _la("la_train", "train", 2, 4096, 12),
        # softmax attention over one 200-token prompt of a two-head layer
        _attn("attn_short_prompt", "fwd", 1, 200, 2, 2),
        # a long prompt, four query heads on each key head, q, k and v out of one projection
        _attn("attn_prompt", "fwd", 1, 16384, 32, 8, fused=True),
        # ragged prompts in one packed batch, small heads, each with its own keys
        _attn("attn_packed_prompts", "fwd", 1, 16411, 12, 12, D=64, seqs=16),
        # a packed training batch of ragged documents with shared key heads
        _attn("attn_train_packed", "train", 1, 8219, 32, 8, seqs=8),
        # one of eight GPUs' share of a training batch, a token more than a power of two
        _attn("attn_train", "train", 2, 4097, 12, 12),
        # one new token for each of 64 running sequences behind 8191 earlier ones: decoding
        _attn("attn_token", "fwd", 64, 1, 32, 8, past=8191),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    fused = rng.random() < 0.4
    if rng.random() < 0.5:
        mode = rng.choice(["fwd", "train", "step"])
        H, K, V = _log(rng, 1, 96), rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        if mode == "step":
            return _la("", mode, _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4]), H, K, V, init=True, fused=fused)
        T = _log(rng, 1, min(262144, (1 << 21) // H))
        B = rng.choice([1, 1, 2, 5])
        return _la("", mode, B, max(1, T // B), H, K, V, fused=fused, init=rng.random() < 0.5,
                   seqs=_log(rng, 2, 64) if B == 1 and rng.random() < 0.6 else 0)
    mode = rng.choice(["fwd", "fwd", "train"])
    Hk, group, D = _log(rng, 1, 16), rng.choice([1, 1, 2, 3, 4, 5, 8]), rng.choice([64, 128, 128])
    if mode == "fwd" and rng.random() < 0.3:  # a few new tokens behind a long past
        B, T, past = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 17]), _log(rng, 1, 8191)
        past = min(past, (1 << 22) // (B * Hk))
        return _attn("", mode, B, T, Hk * group, Hk, D, past=past, fused=fused)
    most = int(math.sqrt((1 << 31) / (Hk * group * (3 if mode == "train" else 1))))
    T, B = _log(rng, 1, min(12288, most)), rng.choice([1, 1, 2, 3])
    seqs = _log(rng, 2, 32) if B == 1 and rng.random() < 0.6 else 0
    past = rng.choice([0, 0, _log(rng, 1, 500)])
    return _attn("", mode, B, max(1, T // B), Hk * group, Hk, D, seqs=seqs, past=past, fused=fused)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=BF16):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    def slices(B, T, *parts):
        """Token arrays [B, T, heads, channels]: each by itself, or views of one projection's output."""
        if not case["fused"]:
            return [normal(B, T, h, c) for h, c in parts]
        wide = normal(B, T, sum(h * c for h, c in parts))
        cut = wide.split([h * c for h, c in parts], -1)
        return [t.unflatten(-1, p) for t, p in zip(cut, parts)]

    s = dict(case)
    B, T = case["B"], case["T"]
    n = case["seqs"] or B
    s["cu_seqlens"] = None
    if case["seqs"]:  # ragged documents between sorted cuts: short and empty ones among them
        cuts = torch.randint(0, T + 1, (n - 1,), generator=gen, device=dev).sort().values
        ends = torch.tensor([0, T], device=dev)
        s["cu_seqlens"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    if case["op"] == "la":
        H, K, V = case["H"], case["K"], case["V"]
        s["q"], s["k"], s["v"] = slices(B, T, (H, K), (H, K), (H, V))
        # the heads' memories reach over one to a thousand tokens
        s["log_decay"] = -torch.exp(torch.rand(H, generator=gen, device=dev) * -math.log(1000.0))
        s["scale"] = K ** -0.5
        s["initial_state"] = normal(n, H, K, V, dtype=torch.float32) if case["init"] else None
        if case["mode"] == "train":
            s["d_out"], s["d_final"] = normal(B, T, H, V), normal(n, H, K, V, dtype=torch.float32)
        return s
    Hq, Hk, D, past = case["Hq"], case["Hk"], case["D"], case["past"]
    s["scale"] = D ** -0.5
    s["cu_seqlens_k"] = None
    if past == 0:
        s["q"], s["k"], s["v"] = slices(B, T, (Hq, D), (Hk, D), (Hk, D))
    else:  # keys and values of earlier tokens in front of each sequence's own
        Tk = T + n * past if case["seqs"] else T + past
        s["q"] = slices(B, T, (Hq, D))[0]
        s["k"], s["v"] = slices(B, Tk, (Hk, D), (Hk, D))
        if case["seqs"]:
            s["cu_seqlens_k"] = s["cu_seqlens"] + torch.arange(n + 1, device=dev, dtype=torch.int32) * past
    if case["mode"] == "train":
        s["d_out"] = normal(B, T, Hq, D)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _chunks(s):
    """The tokens of each sequence in chunks: each chunk's sequence, its first token's place in that
    sequence and its rows (a spare row B T where it has none); each token's place among the chunks."""
    M, dev = s["B"] * s["T"], s["q"].device
    if s["cu_seqlens"] is None:
        first = torch.arange(s["B"], device=dev) * s["T"]
        length = torch.full_like(first, s["T"])
    else:
        cu = s["cu_seqlens"].long()
        first, length = cu[:-1], cu[1:] - cu[:-1]
    count = (length + CHUNK - 1) // CHUNK
    ends = count.cumsum(0)
    c = torch.arange(M // CHUNK + first.numel(), device=dev)  # at most so many
    seq = torch.searchsorted(ends, c, right=True).clamp(max=first.numel() - 1)
    place = (c - (ends - count)[seq]) * CHUNK
    inside = place[:, None] + torch.arange(CHUNK, device=dev)
    rows = torch.where(inside < length[seq][:, None], first[seq][:, None] + inside, M)
    t = torch.arange(M, device=dev)
    n = torch.searchsorted(first + length, t, right=True)
    slot = (ends - count)[n] * CHUNK + t - first[n]
    return length, seq, place, rows, slot


def _plain_la(s):
    """Chunks of 64 tokens: products within a chunk, each chunk's k v^T, and one product over the
    chunks that carries them to the later ones."""
    H, K, V, M = s["H"], s["K"], s["V"], s["B"] * s["T"]
    train = s["mode"] == "train"
    leaf = lambda t: None if t is None else t.detach().float().requires_grad_(train)  # noqa: E731
    q, k, v, g, init = (leaf(s[n]) for n in ("q", "k", "v", "log_decay", "initial_state"))
    length, seq, place, rows, slot = _chunks(s)
    NC, N, dev = seq.numel(), length.numel(), q.device

    def chunked(x):  # [H, NC, CHUNK, channels], zeros where a chunk has no token
        x = torch.cat([x.reshape(M, H, -1), x.new_zeros(1, H, x.shape[-1])])
        return x[rows].permute(2, 0, 1, 3)

    def decay(n):  # exp(n g) for each head, 0 where n is negative
        return torch.exp(g.view(-1, *[1] * n.dim()) * n.clamp(min=0)) * (n >= 0)

    qc, kc, vc = chunked(q), chunked(k), chunked(v)
    i = torch.arange(CHUNK, device=dev)
    held = (length[seq] - place).clamp(0, CHUNK)  # tokens of each chunk
    scores = qc @ kc.transpose(-1, -2) * decay(i[:, None] - i)[:, None]
    added = (kc * decay(held[:, None] - 1 - i)[..., None]).transpose(-1, -2) @ vc  # [H, NC, K, V]
    same = (seq[:, None] == seq) & (place < place[:, None])
    apart = torch.where(same, place[:, None] - place - held, -1)
    enter = (decay(apart) @ added.flatten(2)).view(H, NC, K, V)
    last = torch.where(seq == torch.arange(N, device=dev)[:, None], length[:, None] - place - held, -1)
    final = decay(torch.where(held > 0, last, -1)) @ added.flatten(2)
    final = final.view(H, N, K, V).transpose(0, 1)
    if init is not None:
        enter = enter + decay(place)[..., None, None] * init[seq].transpose(0, 1)
        final = final + decay(length)[..., None, None].transpose(0, 1) * init
    o = scores @ vc + decay(i + 1)[:, None, :, None] * (qc @ enter)
    out = s["scale"] * o.flatten(1, 2)[:, slot].transpose(0, 1).reshape(s["v"].shape)
    if not train:
        return out.to(BF16), final.contiguous()
    leaves = [t for t in (q, k, v, g, init) if t is not None]
    grads = torch.autograd.grad((out, final), leaves, (s["d_out"].float(), s["d_final"]))
    return (out.detach().to(BF16), final.detach().contiguous(), *(t.to(BF16) for t in grads[:3]), *grads[3:])


def _seen(s):
    """Which keys a query sees, [B, Tq, Tk]: of its own sequence, up to its own place from the end."""
    Tq, Tk, dev = s["T"], s["k"].shape[1], s["q"].device
    tq, tk = torch.arange(Tq, device=dev), torch.arange(Tk, device=dev)
    if s["cu_seqlens"] is None:
        return (tk <= tq[:, None] + (Tk - Tq)).expand(s["B"], Tq, Tk)
    cq = s["cu_seqlens"].long()
    ck = cq if s["cu_seqlens_k"] is None else s["cu_seqlens_k"].long()
    nq, nk = (torch.searchsorted(c[1:].contiguous(), t, right=True) for c, t in ((cq, tq), (ck, tk)))
    return ((nq[:, None] == nk) & (tk - ck[1:][nk] <= (tq - cq[1:][nq])[:, None]))[None]


def _plain_attn(s):
    B, T, Hq, Hk, D = s["B"], s["T"], s["Hq"], s["Hk"], s["D"]
    G = Hq // Hk

    def heads(x):  # fp32 [B, Hq, tokens, D]
        return x.float().repeat_interleave(Hq // x.shape[2], 2).transpose(1, 2).contiguous()

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~_seen(s)[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp(min=torch.finfo(torch.float32).tiny)
    o = p @ v
    lse = (top + torch.log(total)).squeeze(-1).transpose(1, 2).contiguous()
    out = o.transpose(1, 2).to(BF16).contiguous()
    if s["mode"] != "train":
        return out, lse
    do = heads(s["d_out"])
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)

    def shared(x):  # the sum over the query heads of each key head
        return x.unflatten(1, (Hk, G)).sum(2).transpose(1, 2).to(BF16).contiguous()

    dq = (ds @ k).mul_(s["scale"]).transpose(1, 2).to(BF16).contiguous()
    return (out, lse, dq, shared((ds.transpose(-1, -2) @ q).mul_(s["scale"])), shared(p.transpose(-1, -2) @ do))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_la(s):
    import chunked_gated_delta_amd as kda
    from chunked_gated_delta_amd.function import kda_linear_attn

    q, k, v, g, init, scale = s["q"], s["k"], s["v"], s["log_decay"], s["initial_state"], s["scale"]
    if s["mode"] == "step":
        out, final = torch.empty(v.shape, dtype=v.dtype, device=v.device), torch.empty_like(init)
        kda.kda_la_step(q, k, v, g, scale, out, initial_state=init, final_state=final)
        return out, final
    if s["mode"] == "fwd":
        return kda_linear_attn(q, k, v, g, scale=scale, initial_state=init, cu_seqlens=s["cu_seqlens"])
    leaves = [t.detach().requires_grad_() for t in (q, k, v, g, init) if t is not None]
    out, final = kda_linear_attn(*leaves[:4], scale=scale, initial_state=None if init is None else leaves[4],
                                 cu_seqlens=s["cu_seqlens"])
    return (out, final, *torch.autograd.grad((out, final), leaves, (s["d_out"], s["d_final"])))


def _own_attn(s):
    from chunked_gated_delta_amd.function import kda_attn

    kw = dict(scale=s["scale"], cu_seqlens=s["cu_seqlens"], cu_seqlens_k=s["cu_seqlens_k"])
    if s["mode"] == "fwd":
        return kda_attn(s["q"], s["k"], s["v"], **kw)
    leaves = [t.detach().requires_grad_() for t in (s["q"], s["k"], s["v"])]
    out, lse = kda_attn(*leaves, **kw)
    return (out, lse, *torch.autograd.grad(out, leaves, s["d_out"]))


def run(state):
    if own:
        return (_own_la if state["op"] == "la" else _own_attn)(state)
    return (_plain_la if state["op"] == "la" else _plain_attn)(state)


def work(case):
    """Each input read once, each output written once; operations of the recurrence, and of the pairs
    of a query and a key that it sees (packed sequences: as many as evenly drawn cuts leave)."""
    M, n, train = case["B"] * case["T"], case["seqs"] or case["B"], case["mode"] == "train"
    if case["op"] == "la":
        H, K, V = case["H"], case["K"], case["V"]
        tokens = M * H * 2 * ((2 * K + 2 * V) + ((2 * K + 2 * V) if train else 0))
        states = n * H * K * V * 4 * (1 + case["init"]) * (2 if train else 1)
        return {"bytes": tokens + states + H * 4 * (2 if train else 1),
                "flops": M * H * K * V * 4 * (4 if train else 1)}
    T, Hq, Hk, D, past = case["T"], case["Hq"], case["Hk"], case["D"], case["past"]
    pairs = T * T / (n + 1) if case["seqs"] else case["B"] * T * (T + 1) / 2
    pairs += M * past
    keys = M + n * past
    tokens = 2 * D * (2 * M * Hq + 2 * keys * Hk)
    return {"bytes": tokens * (2 if train else 1) + M * Hq * 4,
            "flops": pairs * Hq * D * (14 if train else 4)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _bounds(s, name, total):
    if s[name] is None:
        return [(b * total, (b + 1) * total) for b in range(s["B"])]
    cu = s[name].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_la(s):
    """Sequence by sequence, its state carried from one block of tokens to the next; a token's output
    is the sum over the block's earlier tokens and the state that entered the block."""
    H, K, V, block = s["H"], s["K"], s["V"], 256
    train, dev = s["mode"] == "train", s["q"].device
    seqs = _bounds(s, "cu_seqlens", s["T"])
    leaf = lambda t: t.double().detach().requires_grad_(train)  # noqa: E731
    q, k, v, g = (leaf(s[n]) for n in ("q", "k", "v", "log_decay"))
    zero = torch.zeros(len(seqs), H, K, V, dtype=torch.float64, device=dev)
    init = leaf(zero if s["initial_state"] is None else s["initial_state"])
    qr, kr, vr = (x.reshape(-1, H, x.shape[-1]).transpose(0, 1) for x in (q, k, v))
    outs, finals = [], []
    for n, (lo, hi) in enumerate(seqs):
        state = init[n]
        for a in range(lo, hi, block):
            z = min(a + block, hi)
            x, y, w = qr[:, a:z], kr[:, a:z], vr[:, a:z]
            t = torch.arange(z - a, device=dev, dtype=torch.float64)
            gap = t[:, None] - t
            within = torch.exp(g[:, None, None] * gap.clamp(min=0)).tril()
            reach = torch.exp(g[:, None] * (t + 1))[..., None]
            outs.append((x @ y.transpose(1, 2).contiguous() * within) @ w + (x * reach) @ state)
            left = torch.exp(g[:, None] * (z - a - 1 - t))[..., None]
            state = torch.exp(g * (z - a))[:, None, None] * state + (y * left).transpose(1, 2).contiguous() @ w
        finals.append(state)
    out = s["scale"] * torch.cat(outs, 1).transpose(0, 1).reshape(s["v"].shape)
    final = torch.stack(finals)
    if not train:
        return out, final
    leaves = [q, k, v, g] + ([init] if s["init"] else [])
    grads = torch.autograd.grad((out, final), leaves, (s["d_out"].double(), s["d_final"].double()))
    return (out.detach(), final.detach(), *grads)


def _exact_attn(s):
    """Sequence by sequence and head by head: the softmax of the scores that a query sees."""
    Hq, Hk, D, train = s["Hq"], s["Hk"], s["D"], s["mode"] == "train"
    flat = lambda t: t.double().reshape(-1, t.shape[2], D).transpose(0, 1)  # noqa: E731
    q, k, v = flat(s["q"]), flat(s["k"]), flat(s["v"])
    bq = _bounds(s, "cu_seqlens", s["T"])
    bk = bq if s["past"] == 0 else _bounds(s, "cu_seqlens_k", s["k"].shape[1])
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = flat(s["d_out"]) if train else None
    for (lo, hi), (a, z) in zip(bq, bk):
        hidden = torch.ones(hi - lo, z - a, dtype=torch.bool, device=q.device).triu(z - a - (hi - lo) + 1)
        for h in range(Hq if hi > lo else 0):
            x, y, w = q[h, lo:hi], k[h * Hk // Hq, a:z], v[h * Hk // Hq, a:z]
            score = torch.where(hidden, -math.inf, s["scale"] * (x @ y.T))
            sums = torch.logsumexp(score, -1)
            p = torch.exp(score - sums[:, None])
            out[h, lo:hi], lse[h, lo:hi] = p @ w, sums
            if train:
                d = do[h, lo:hi]
                ds = p * (d @ w.T - (d * out[h, lo:hi]).sum(-1, keepdim=True)) * s["scale"]
                dq[h, lo:hi] = ds @ y
                dk[h * Hk // Hq, a:z] += ds.T @ x
                dv[h * Hk // Hq, a:z] += p.T @ d
    shape = lambda t, like: t.transpose(0, 1).reshape(like.shape)  # noqa: E731
    res = (shape(out, s["q"]), lse.T.reshape(s["q"].shape[:3]))
    return (*res, shape(dq, s["q"]), shape(dk, s["k"]), shape(dv, s["v"])) if train else res


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_la if case["op"] == "la" else _exact_attn)(s)
