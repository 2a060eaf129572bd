"""Gradients made outside autograd, tied to what they were made from (causal_scaled_dot_gb300/autograd.py)."""
import pytest
import torch
from torch.autograd import forward_ad

from causal_scaled_dot_gb300.autograd import refuse_tangents, tied


class Cube(torch.autograd.Function):
    """w x^3, whose gradients no operation of torch's records."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return w * x ** 3

    @staticmethod
    def backward(ctx, up):
        x, w = ctx.saved_tensors
        with torch.no_grad():
            dx, dw = 3 * w * x * x * up, x ** 3 * up
        return (tied(dx, up, x, w), tied(dw, up, x)) if torch.is_grad_enabled() else (dx, dw)


def leaves(x=True, w=True):
    return torch.tensor([2.0, -1.0], requires_grad=x), torch.tensor([3.0, 0.5], requires_grad=w)


def test_a_penalty_under_a_constant_upstream_is_refused():
    x, w = leaves(w=False)
    y = Cube.apply(x, w).sum()
    g, = torch.autograd.grad(y, x, create_graph=True)
    assert torch.equal(g, 3 * w * x.detach() ** 2)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (y + g.square().sum()).backward()


def test_an_upstream_that_requires_a_gradient_is_refused():
    x, w = leaves()
    up = torch.ones(2, requires_grad=True)
    g, = torch.autograd.grad(Cube.apply(x.detach(), w), w, up, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.sum().backward()


def test_what_depends_on_nothing_is_a_constant():
    x, w = leaves(x=False)
    y = Cube.apply(x, w).sum()
    g, = torch.autograd.grad(y, w, create_graph=True)  # x^3: no w in it
    assert not g.requires_grad
    (y + g.square().sum()).backward()
    assert torch.equal(w.grad, x ** 3)


def test_first_order_is_as_it_was():
    x, w = leaves()
    want = torch.autograd.grad(Cube.apply(x, w).sum(), (x, w))
    for g, e in zip(torch.autograd.grad(Cube.apply(x, w).sum(), (x, w), create_graph=True), want):
        assert torch.equal(g, e) and not e.requires_grad
        g.mul_(2)  # an ordinary tensor
    Cube.apply(x, w).sum().backward(create_graph=True)
    Cube.apply(x, w).sum().backward()
    assert torch.equal(x.grad, 2 * want[0]) and torch.equal(w.grad, 2 * want[1])
    with torch.no_grad():
        x.grad.zero_()


def test_tangents_are_refused():
    t = torch.ones(3)
    refuse_tangents(t, None)
    with forward_ad.dual_level():
        refuse_tangents(t, None)
        with pytest.raises(ValueError, match="tangent"):
            refuse_tangents(t, None, forward_ad.make_dual(t, t))
    refuse_tangents(t)
