"""The rotation as a node of torch's graph, on the host: the kernel is replaced by the
plain form in torch, which leaves the binding's own part, what derivatives follow."""
from __future__ import annotations

import pytest
import torch
import torch.autograd.forward_ad as fwad

import token_decode_attention_gb300 as dattn
from token_decode_attention_gb300 import _native

from . import _q8


@pytest.fixture
def calls(monkeypatch):
    """The rotations that reach the kernel's place: (gradient, contiguous, aligned)."""
    seen = []

    def plain(x, out, positions, rope_dims, rope_base, traditional, scaling, gradient, stream):
        assert not out.requires_grad
        seen.append((gradient, x.is_contiguous(), x.data_ptr() % 16 == 0 and x.data_ptr() != 0))
        y = _q8.rotate(x.detach().numpy(), positions.numpy(), rope_dims, rope_base, traditional, scaling, gradient)
        out.numpy()[...] = y     # as the kernel does, past torch
    monkeypatch.setattr(_native, "_rope", plain)
    return seen


def rotated(x, p, gradient=False):
    return torch.from_numpy(_q8.rotate(x.detach().numpy(), p.numpy(), gradient=gradient)).float()


X, T = torch.randn((5, 2, 32), generator=torch.Generator().manual_seed(1)), torch.ones((5, 2, 32))
T[1] = -2.0
P = torch.arange(5, dtype=torch.int32) * 7


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("requires", [False, True])
def test_forward_mode_rotates_the_tangent(calls, gradient, requires):
    x = X.clone().requires_grad_(requires)
    with fwad.dual_level():
        y = dattn.rope(fwad.make_dual(x, T), P, gradient=gradient)
        value, tangent = fwad.unpack_dual(y)
        assert tangent is not None and torch.equal(value.detach(), rotated(X, P, gradient))
        assert torch.equal(tangent, rotated(T, P, gradient))
    with fwad.dual_level(), torch.no_grad():   # which does not turn forward mode off
        y = dattn.rope(fwad.make_dual(x, T), P, gradient=gradient)
        assert torch.equal(fwad.unpack_dual(y).tangent, rotated(T, P, gradient))
    assert all(c and a for _, c, a in calls)


def test_tangents_of_any_layout(calls):
    wide = torch.randn((5, 2, 64))
    for t in (T[:1].expand(5, 2, 32)[:, :, :], wide[:, :, 1:33], wide[:, :, ::2], torch._efficientzerotensor((5, 2, 32))):
        with fwad.dual_level():
            y = dattn.rope(fwad.make_dual(X, t), P)
            assert torch.equal(fwad.unpack_dual(y).tangent, rotated(t.clone(), P))
    assert all(c and a for _, c, a in calls)


def test_forward_over_reverse(calls):
    # the derivative of x -> R^T (3 (R x)^2) along T is R^T (6 (R x) (R T))
    x = X.clone().requires_grad_()
    with fwad.dual_level():
        y = dattn.rope(fwad.make_dual(x, T), P)
        g, = torch.autograd.grad((y ** 3).sum(), x, create_graph=True)
        tangent = fwad.unpack_dual(g).tangent
    want = rotated(6 * rotated(X, P) * rotated(T, P), P, True)
    # fp32 products of terms below 200, rounded some six times on either side
    assert float((tangent.detach() - want).abs().max()) <= 200 * 12 * 2.0 ** -24


def test_a_tangent_refuses_out_and_stream(calls):
    with fwad.dual_level():
        d = fwad.make_dual(X, T)
        with pytest.raises(ValueError, match="gradient"):
            dattn.rope(d, P, out=torch.empty_like(X))
        with pytest.raises(ValueError, match="gradient"):
            dattn.rope(d, P, stream=object())
    assert not calls


def test_writing_to_out_counts_as_a_change_in_place(calls):
    x, w = X.clone(), torch.ones_like(X, requires_grad=True)
    y = (w * x).sum()            # the graph keeps x for w's gradient
    before = x._version
    dattn.rope(x, P, out=x)
    assert x._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    out = torch.empty_like(X)
    before = out._version
    dattn.dattn_rope(X, out, P)
    assert out._version > before
    with torch.inference_mode():
        out = torch.empty_like(X)
        dattn.rope(X, P, out=out)    # such a tensor counts no changes


def test_the_call_without_a_graph_refuses_to_lose_a_gradient(calls):
    x, out = X.clone().requires_grad_(), torch.empty_like(X)
    with pytest.raises(ValueError, match="gradient"):
        dattn.dattn_rope(x, out, P)
    with pytest.raises(ValueError, match="gradient"):
        dattn.rope(X, P, out=torch.empty_like(X).requires_grad_())
    with fwad.dual_level():
        with pytest.raises(ValueError, match="gradient"):
            dattn.dattn_rope(fwad.make_dual(X, T), out, P)
    assert not calls
    with torch.no_grad():
        dattn.dattn_rope(x, out, P)
    assert torch.equal(out, rotated(X, P))


def test_neither_pass_is_captured(calls, monkeypatch):
    x = X.clone().requires_grad_()
    y = dattn.rope(x, P)
    monkeypatch.setattr(_native, "_captured", lambda t: True, raising=False)
    with pytest.raises(ValueError, match="captured"):
        dattn.rope(x, P)
    # the forward pass was an ordinary call, its backward pass is being captured
    with pytest.raises(ValueError, match="captured"):
        y.sum().backward()
    assert x.grad is None
    with torch.no_grad():
        dattn.rope(x, P, gradient=True)
    monkeypatch.undo()
