"""The differentiable wrappers of the operators around the core on the GPU: what autograd hands them
and takes from them.  Values are compared with test_gpu_around.py's tolerances or bit for bit."""

import pytest
import torch

import chunked_gated_delta_amd as kda
from chunked_gated_delta_amd.function import kda_chunk, kda_glr, kda_qk_norm_rope, kda_short_conv
from test_gpu_around import DEV, Rand, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ops(ty):
    """Per operator: the call and its inputs."""
    r = Rand(90)
    a = lambda *s, dtype=torch.float32, std=1.0: r(*s, dtype=dtype, std=std).to(DEV)  # noqa: E731
    pos, f = torch.arange(70, dtype=torch.int32, device=DEV)[None], torch.full((8,), 0.3, dtype=torch.float64, device=DEV)
    bf = torch.bfloat16
    return {
        "glr": (lambda x, g, al, dt, i: kda_glr(x, g, al, dt, initial_state=i),
                [a(1, 70, 2, 32, dtype=ty), a(1, 70, 2, 32, dtype=ty), a(2), a(2, 32), a(1, 2, 32)]),
        "conv": (lambda x, w, b, i: kda_short_conv(x, w, b, initial_state=i),
                 [a(1, 70, 64, dtype=ty), a(64, 4), a(64), a(1, 3, 64, dtype=ty)]),
        "qk": (lambda q, k, qw, kw: kda_qk_norm_rope(q, k, pos, f, q_weight=qw, k_weight=kw, norm="rms"),
               [a(1, 70, 3, 32, dtype=ty), a(1, 70, 2, 32, dtype=ty), 1 + a(32, std=0.2), 1 + a(32, std=0.2)]),
        "chunk": (lambda q, k, v, g, b, al, dt, i: kda_chunk(q, k, v, g, b, al, dt, initial_state=i),
                  [*(a(1, 70, 2, 64, dtype=bf) for _ in range(4)), a(1, 70, 2, dtype=bf), a(2), a(2, 64),
                   a(1, 2, 64, 64, std=0.1)]),
    }


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("op", ["glr", "conv", "qk", "chunk"])
def test_gradients_through_a_cat_behind_an_odd_piece(op, ty):
    """The same gradients, bit for bit, whether they arrive aligned or one element off."""
    say(op, ty)
    call, t = ops(ty)[op]
    t = [v.requires_grad_() for v in t]
    outs = call(*t)
    r = Rand(91)
    d = [r(*o.shape, dtype=o.dtype).to(DEV) for o in outs]
    want = torch.autograd.grad(outs, t, d, retain_graph=True)
    whole = [torch.cat([o.new_zeros(1), o.flatten()]) for o in outs]
    got = torch.autograd.grad(whole, t, [torch.cat([x.new_zeros(1), x.flatten()]) for x in d])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("reuse", [False, True])
def test_the_core_trains_on_rows_of_the_norm_and_rotation(reuse):
    """kda_qk_norm_rope, then kda_chunk without a norm of its own: the bits of the library's calls with
    FLAG_NO_QK_NORM, and near kda_chunk's own norm of the same rows where nothing is rotated."""
    r, T, H, K = Rand(92), 130, 2, 64
    a = lambda *s, dtype=torch.bfloat16, std=1.0: r(*s, dtype=dtype, std=std).to(DEV)  # noqa: E731
    q, k, v, g, b = a(1, T, H, K), a(1, T, H, K), a(1, T, H, K), a(1, T, H, K), a(1, T, H)
    al, dt = a(H, dtype=torch.float32, std=0.5), a(H, K, dtype=torch.float32, std=0.1)
    cu = torch.tensor([0, 70, 130], dtype=torch.int32, device=DEV)
    leaves = [t.requires_grad_() for t in (q, k, v, g, b, al, dt)]
    pos, f = torch.arange(T, dtype=torch.int32, device=DEV)[None], torch.full((8,), 0.3, dtype=torch.float64, device=DEV)
    d, df = a(1, T, H, K), a(2, H, K, K, dtype=torch.float32)
    qn, kn = kda_qk_norm_rope(q, k, pos, f)
    out, fin = kda_chunk(qn, kn, v, g, b, al, dt, cu_seqlens=cu, reuse_records=reuse, qk_normalized=True)
    got = torch.autograd.grad((out, fin), [qn, kn, *leaves[2:]], (d, df))

    with torch.no_grad():
        o2, f2 = torch.empty_like(out), torch.empty_like(fin)
        ws = torch.empty(kda.kda_bwd_workspace_size(T, H, 2), dtype=torch.uint8, device=DEV)
        kda.kda_fwd_ex(qn, kn, v, g, b, K ** -0.5, o2, ws, al, dt, -5.0, None, f2, cu, flags=kda.FLAG_NO_QK_NORM)
        assert kda.kda_workspace_faults(ws) == 0
        want = [torch.empty_like(t) for t in (qn, kn, *leaves[2:])]
        kda.kda_bwd_ex(qn, kn, v, g, b, K ** -0.5, d, *want, ws, al, dt, -5.0, None, df, None, cu,
                       flags=kda.FLAG_NO_QK_NORM)
    assert torch.equal(out, o2) and torch.equal(fin, f2)
    assert all(torch.equal(x, y) for x, y in zip(got, want))

    # unrotated, the two ways differ by the rounding of the normed rows to bf16: 2^-8 of each of the two
    # operands, forward and again backward, against the core's own parity bound of 1e-2 (rel. 2-norm)
    qn, kn = kda_qk_norm_rope(q, k)
    pair = [kda_chunk(qn, kn, v, g, b, al, dt, cu_seqlens=cu, qk_normalized=True),
            kda_chunk(q, k, v, g, b, al, dt, cu_seqlens=cu)]
    grads = [torch.autograd.grad(p, leaves, (d, df)) for p in pair]
    for x, y in zip((*pair[0], *grads[0]), (*pair[1], *grads[1])):
        assert ((x.double() - y.double()).norm() / y.double().norm()).item() <= 1e-2 + 4 * 2.0 ** -8
