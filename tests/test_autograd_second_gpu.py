"""Gradients of native.attention_trainable that are differentiated again: refused, as they depend on q, k and v."""
import pytest
import torch

from causal_scaled_dot_gb300 import native
from tests.cache_util import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture
def qkv():
    return [rows((1, H, 40, 64), 3 + H).cuda().requires_grad_() for H in (4, 2, 2)]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_penalty_on_a_gradient(which, qkv):
    y = native.attention_trainable(*qkv).float().sum()
    g, = torch.autograd.grad(y, qkv[which], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (y + g.float().square().sum()).backward()


def test_an_upstream_gradient_that_requires_one(qkv):
    o = native.attention_trainable(*(t.detach() for t in qkv[:2]), qkv[2])
    g, = torch.autograd.grad(o, qkv[2], torch.ones_like(o).requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.float().sum().backward()


def test_the_first_derivatives_are_the_same(qkv):
    want = torch.autograd.grad(native.attention_trainable(*qkv).float().sum(), qkv)
    got = torch.autograd.grad(native.attention_trainable(*qkv).float().sum(), qkv, create_graph=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not b.requires_grad
    native.attention_trainable(*qkv).float().sum().backward(create_graph=True)
    for t, b in zip(qkv, want):
        assert torch.equal(t.grad, b)
        t.grad = None


def test_the_values_gradient_does_not_depend_on_the_values(qkv):
    q, k, v = qkv[0].detach(), qkv[1].detach(), qkv[2]
    y = native.attention_trainable(q, k, v).float().sum()
    g, = torch.autograd.grad(y, v, create_graph=True)
    assert not g.requires_grad
    (y + g.float().square().sum()).backward()
    assert torch.equal(v.grad, g)
