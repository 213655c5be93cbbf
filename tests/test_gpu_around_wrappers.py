"""The differentiable wrappers of the operators around the core on the GPU: what autograd hands them
and takes from them.  Values are compared with test_gpu_around.py's tolerances or bit for bit."""

import pytest
import torch

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
