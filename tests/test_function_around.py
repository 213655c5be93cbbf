"""The differentiable wrappers of the operators around the core, on the CPU: what they hand to the
library's calls, which are replaced here, and what autograd sees of them."""

import weakref

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from chunked_gated_delta_amd import function as F

CALLS = ("kda_glr_fwd", "kda_glr_bwd", "kda_conv_fwd", "kda_conv_bwd", "kda_qk_rope_fwd", "kda_qk_rope_bwd")


@pytest.fixture
def library(monkeypatch):
    """The arguments of every call, by its name; nothing is computed."""
    seen = {}
    for name in CALLS:
        monkeypatch.setattr(F, name, lambda *a, _name=name, **k: seen.setdefault(_name, []).append(a))
    return seen


def inputs(ty=torch.bfloat16):
    """Per operator: the call, and its inputs that may be differentiated, by name."""
    x = torch.randn(1, 6, 2, 8, dtype=ty)
    pos, f = torch.zeros(1, 6, dtype=torch.int32), torch.ones(4, dtype=torch.float64)
    return {
        "glr": (lambda x, raw_gate, A_log, dt_bias, initial_state: F.kda_glr(x, raw_gate, A_log, dt_bias,
                                                                             initial_state=initial_state),
                dict(x=x, raw_gate=torch.randn(1, 6, 2, 8, dtype=ty), A_log=torch.randn(2), dt_bias=torch.randn(2, 8),
                     initial_state=torch.randn(1, 2, 8))),
        "conv": (lambda x, weight, bias, initial_state: F.kda_short_conv(x, weight, bias, initial_state=initial_state),
                 dict(x=torch.randn(1, 6, 16, dtype=ty), weight=torch.randn(16, 4), bias=torch.randn(16),
                      initial_state=torch.randn(1, 3, 16, dtype=ty))),
        "qk": (lambda q, k, q_weight, k_weight: F.kda_qk_norm_rope(q, k, pos, f, q_weight=q_weight, k_weight=k_weight),
               dict(q=x, k=torch.randn(1, 6, 1, 8, dtype=ty), q_weight=torch.randn(8), k_weight=torch.randn(8))),
    }


NAMES = [(op, n) for op, (_, t) in inputs().items() for n in t]


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("op,name", NAMES)
def test_a_tangent_is_refused_not_dropped(op, name, grad, library):
    """These operators have no forward-mode derivative: an input with a tangent is an error, with and
    without a graph to record, and a call without one inside the same level is not."""
    call, t = inputs()[op]
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        call(**t)
        t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
        with pytest.raises(NotImplementedError, match="jvp"):
            call(**t)
    assert not any(o.requires_grad for o in call(**inputs()[op][1]))


def at_odd_place(t):
    """The same values, contiguous, one element behind an aligned address."""
    flat = torch.cat([t.new_zeros(1), t.flatten()])
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("op,ty", [(op, ty) for op in ("glr", "conv", "qk") for ty in (torch.bfloat16, torch.float32)])
def test_gradients_may_arrive_at_any_address(op, ty, library):
    """The gradient of a piece of a cat is a view at the piece's offset: contiguous and not aligned.
    The kernels' loads are of up to 16 bytes."""
    call, t = inputs(ty)[op]
    outs = call(**{n: v.requires_grad_() for n, v in t.items()})
    grads = [torch.randn_like(o) for o in outs]
    torch.autograd.backward(outs, [at_odd_place(g) for g in grads])
    name, first, second = {"glr": ("kda_glr_bwd", 3, 13), "conv": ("kda_conv_bwd", 2, 9),
                           "qk": ("kda_qk_rope_bwd", 2, 3)}[op]
    (args,) = library[name]
    for got, want in zip((args[first], args[second]), grads):
        assert torch.equal(got, want) and got.is_contiguous() and got.data_ptr() % 16 == 0
    # as autograd itself hands them out
    library.clear()
    out = call(**t)[0]
    torch.cat([out.new_zeros(1), out.flatten()]).sum().backward()
    (args,) = library[name]
    assert (args[first] == 1).all() and args[first].shape == out.shape and args[first].data_ptr() % 16 == 0


def test_gradients_of_the_core_may_arrive_at_any_address(monkeypatch):
    seen = []
    monkeypatch.setattr(F, "kda_fwd_ex", lambda *a, **k: None)
    monkeypatch.setattr(F, "kda_bwd_ex", lambda *a, **k: seen.append((a[6], k["d_final"])))
    q, k, v, g = (torch.randn(1, 64, 1, 64, dtype=torch.bfloat16).requires_grad_() for _ in range(4))
    outs = F.kda_chunk(q, k, v, g, torch.randn(1, 64, 1, dtype=torch.bfloat16), torch.zeros(1), torch.zeros(1, 64))
    grads = [torch.randn_like(o) for o in outs]
    torch.autograd.backward(outs, [at_odd_place(d) for d in grads])
    for got, want in zip(seen[0], grads):
        assert got.data_ptr() % 16 == 0 and torch.equal(got, want)


def test_the_recurrences_states_are_saved_tensors(library):
    """What the forward leaves for the backward is seen by saved-tensor hooks and freed with the graph,
    also while an output is still held."""
    call, t = inputs()["glr"]
    size = F.kda_glr_states_size(6, 2, 8)
    packed = []

    def pack(v):
        packed.append(v)
        return v

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda v: v):
        outs = call(**{n: v.requires_grad_() for n, v in t.items()})
    assert [v.numel() for v in packed if v.dtype is torch.uint8] == [size]
    packed.clear()
    outs = call(**t)
    (_, states), _ = library["kda_glr_fwd"][-1][8:10], library.clear()
    ref = weakref.ref(states.untyped_storage())
    outs[0].float().sum().backward()
    (args,) = library["kda_glr_bwd"]
    assert args[2].data_ptr() == states.data_ptr()
    del states, args
    library.clear()
    assert ref() is None and outs[0] is not None


def test_frequencies_that_want_a_derivative_are_refused(library):
    """The rotation's frequencies have no gradient: asked for one, the call fails rather than leave it out."""
    q, f, pos = torch.randn(1, 6, 2, 8, dtype=torch.bfloat16), torch.ones(4, dtype=torch.float64), torch.zeros(1, 6).int()
    with pytest.raises(ValueError, match="inv_freq"):
        F.kda_qk_norm_rope(q, q, pos, f.clone().requires_grad_())
    with torch.no_grad():
        F.kda_qk_norm_rope(q, q, pos, f.clone().requires_grad_())
    with forward_ad.dual_level(), pytest.raises(NotImplementedError, match="jvp"):
        F.kda_qk_norm_rope(q, q, pos, forward_ad.make_dual(f, f))


@pytest.mark.parametrize("reuse", [False, True])
def test_the_core_takes_rows_that_are_normed_already(reuse, monkeypatch):
    """qk_normalized is the library's flag in both directions, beside those of the records."""
    flags = []
    monkeypatch.setattr(F, "kda_fwd_ex", lambda *a, **k: flags.append(k["flags"]))
    monkeypatch.setattr(F, "kda_bwd_ex", lambda *a, **k: flags.append(k["flags"]))
    q, k, v, g = (torch.randn(1, 64, 1, 64, dtype=torch.bfloat16).requires_grad_() for _ in range(4))
    rest = (torch.randn(1, 64, 1, dtype=torch.bfloat16), torch.zeros(1), torch.zeros(1, 64))
    for normed, bit in ((False, 0), (True, F.FLAG_NO_QK_NORM)):
        flags.clear()
        F.kda_chunk(q, k, v, g, *rest, reuse_records=reuse, qk_normalized=normed)[0].float().sum().backward()
        assert flags == [bit | (F.FLAG_KEEP_RECORDS if reuse else 0), bit | (F.FLAG_REUSE_RECORDS if reuse else 0)]
