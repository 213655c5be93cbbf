"""The differentiable wrappers of the token mixers on the CPU: what they hand to the library's calls,
which are replaced here, and what autograd sees of them."""

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from chunked_gated_delta_amd import function as F
from test_function_around import at_odd_place


@pytest.fixture
def library(monkeypatch):
    """The arguments of every call, by its name; nothing is computed."""
    seen = {}
    for name in ("kda_la_fwd", "kda_la_bwd", "kda_attn_fwd", "kda_attn_bwd"):
        monkeypatch.setattr(F, name, lambda *a, _name=name, **k: seen.setdefault(_name, []).append(a))
    return seen


def inputs():
    bf = lambda *s: torch.randn(*s, dtype=torch.bfloat16)  # noqa: E731
    return {"la": (lambda q, k, v, g, i: F.kda_linear_attn(q, k, v, g, initial_state=i),
                   dict(q=bf(1, 6, 2, 64), k=bf(1, 6, 2, 64), v=bf(1, 6, 2, 128), g=-torch.rand(2), i=torch.randn(1, 2, 64, 128))),
            "attn": (lambda q, k, v: F.kda_attn(q, k, v), dict(q=bf(1, 6, 4, 64), k=bf(1, 6, 2, 64), v=bf(1, 6, 2, 64)))}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("op,name", [(op, n) for op, (_, t) in inputs().items() for n in t])
def test_a_tangent_is_refused_not_dropped(op, name, grad, library):
    call, t = inputs()[op]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        call(**t)
        t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
        with pytest.raises(NotImplementedError, match="jvp"):
            call(**t)
    assert not any(o.requires_grad for o in call(**inputs()[op][1]))


@pytest.mark.parametrize("op", ["la", "attn"])
def test_gradients_may_arrive_at_any_address(op, library):
    call, t = inputs()[op]
    outs = call(**{n: v.requires_grad_() for n, v in t.items()})
    grads = [torch.randn_like(o) for o in outs]
    torch.autograd.backward(outs, [at_odd_place(g) for g in grads])
    name, places = {"la": ("kda_la_bwd", (5, 12)), "attn": ("kda_attn_bwd", (7, 12))}[op]
    (args,) = library[name]
    for i, want in zip(places, grads):
        assert torch.equal(args[i], want) and args[i].is_contiguous() and args[i].data_ptr() % 16 == 0


def test_what_is_not_asked_for_is_not_computed(library):
    call, t = inputs()["la"]
    call(**t)
    outs = call(**(t | dict(q=t["q"].clone().requires_grad_())))
    outs[0].sum().backward()
    (args,) = library["kda_la_bwd"]
    assert args[10] is None and args[13] is None  # d_log_decay, d_initial_state
    call, t = inputs()["attn"]
    call(**t)
    call(**(t | dict(q=t["q"].clone().requires_grad_())))
    plain, train = library["kda_attn_fwd"]
    assert plain[7] is None and train[7].shape == t["q"].shape  # out_lo is for a backward


def test_gradients_are_contiguous_whatever_the_inputs_strides(library):
    wide = torch.randn(1, 6, 4 * 64 + 2 * 64 * 2, dtype=torch.bfloat16).requires_grad_()
    q, k, v = wide.split([256, 128, 128], -1)
    F.kda_attn(q.unflatten(-1, (4, 64)), k.unflatten(-1, (2, 64)), v.unflatten(-1, (2, 64)))[0].sum().backward()
    (args,) = library["kda_attn_bwd"]
    assert not args[0].is_contiguous() and all(args[i].is_contiguous() for i in (7, 8, 9, 10))


def test_offsets_of_keys_alone_are_refused(library):
    q = inputs()["attn"][1]["q"]
    with pytest.raises(ValueError, match="cu_seqlens"):
        F.kda_attn(q, q, q, cu_seqlens_k=torch.zeros(2, dtype=torch.int32))
    F.kda_attn(q, q, q, cu_seqlens=torch.tensor([0, 6], dtype=torch.int32))
    (args,) = library["kda_attn_fwd"]
    assert args[8] is args[9] and args[3] == 64 ** -0.5  # the queries' offsets are the keys' too; the default scale
