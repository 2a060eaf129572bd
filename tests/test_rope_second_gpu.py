"""Gradients of rotary positions and norms that are differentiated again: refused where they depend on what requires a
gradient, constants where they do not."""
import pytest
import torch

from causal_scaled_dot_gb300.rotary import Rotary
from tests.cache_util import rows
from tests.test_rope_gpu import weights

pytestmark = pytest.mark.gpu
D, S = 64, 12


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def heads_of(x):
    h = x.unflatten(2, (4, D)).transpose(1, 2)
    return h[:, :2], h[:, 2:3]


def outputs(how, x, q_norm, k_norm):
    """q and k [1, H, S, D] by either call."""
    r = Rotary.from_base(D)
    if how == "heads":
        return r.heads(x, 2, 1, q_norm=q_norm, k_norm=k_norm)[:2]
    return r.rotate(*heads_of(x), q_norm=q_norm, k_norm=k_norm)


def total(*ts):
    """Linear in each: a constant upstream gradient."""
    return sum(t.float().sum() for t in ts)


@pytest.fixture
def x():
    return rows((1, S, 4 * D), 2).cuda()


@pytest.fixture
def w():
    return [t.cuda() for t in weights(D, torch.float32)]


@pytest.mark.parametrize("how", ["heads", "rotate"])
@pytest.mark.parametrize("frozen", [False, True])
def test_a_penalty_on_the_inputs_gradient(how, frozen, x, w):
    """With a norm it depends on the input (and the weight), under a constant upstream gradient too."""
    x.requires_grad_()
    for t in w:
        t.requires_grad_(not frozen)
    y = total(*outputs(how, x, *w))
    g, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (y + g.float().square().sum()).backward()


@pytest.mark.parametrize("how", ["heads", "rotate"])
@pytest.mark.parametrize("which", [0, 1])
def test_a_penalty_on_a_weights_gradient(how, which, x, w):
    x.requires_grad_()
    w[which].requires_grad_()
    y = total(*outputs(how, x, *w))
    g, = torch.autograd.grad(y, w[which], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (y + g.square().sum()).backward()


@pytest.mark.parametrize("how", ["heads", "rotate"])
def test_a_weights_gradient_does_not_depend_on_the_weight(how, x, w):
    w[0].requires_grad_()
    want, = torch.autograd.grad(total(*outputs(how, x, *w)), w[0])
    y = total(*outputs(how, x, *w))
    g, = torch.autograd.grad(y, w[0], create_graph=True)
    assert not g.requires_grad and torch.equal(g, want)
    (y + g.square().sum()).backward()
    assert torch.equal(w[0].grad, want)


@pytest.mark.parametrize("how", ["heads", "rotate"])
def test_without_a_norm_the_gradient_is_a_constant(how, x):
    x.requires_grad_()
    y = total(*outputs(how, x, None, None))
    g, = torch.autograd.grad(y, x, create_graph=True)
    assert not g.requires_grad
    (y + g.float().square().sum()).backward()
    assert torch.equal(x.grad, g)


def test_each_of_q_and_k_by_itself(x, w):
    """q normed, k not: k's gradient is a constant, q's is not."""
    q, k = (t.detach().requires_grad_() for t in heads_of(x))
    y = total(*Rotary.from_base(D).rotate(q, k, q_norm=w[0]))
    gq, gk = torch.autograd.grad(y, (q, k), create_graph=True)
    assert gq.requires_grad and not gk.requires_grad
    (y + gk.float().square().sum()).backward(inputs=[k])
    assert torch.equal(k.grad, gk)


@pytest.mark.parametrize("how", ["heads", "rotate"])
@pytest.mark.parametrize("norm", [False, True])
def test_an_upstream_gradient_that_requires_one(how, norm, x, w):
    x.requires_grad_()
    q, k = outputs(how, x, *(w if norm else (None, None)))
    up = [torch.ones_like(q).requires_grad_(), torch.ones_like(k)]
    g, = torch.autograd.grad((q, k), x, up, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.float().sum().backward()


@pytest.mark.parametrize("how", ["heads", "rotate"])
def test_the_first_derivatives_are_the_same(how, x, w):
    """With create_graph, with tensors that hooks moved, and in a checkpoint, which lets what is saved be unpacked once."""
    from torch.utils.checkpoint import checkpoint
    leaves = [x.requires_grad_(), *(t.requires_grad_() for t in w)]
    want = torch.autograd.grad(total(*outputs(how, *leaves)), leaves)
    with torch.autograd.graph.save_on_cpu():
        y = total(*outputs(how, *leaves))
    moved = torch.autograd.grad(y, leaves, create_graph=True)
    again = torch.autograd.grad(checkpoint(lambda *t: total(*outputs(how, *t)), *leaves, use_reentrant=False), leaves)
    plain = torch.autograd.grad(checkpoint(lambda *t: total(*outputs(how, *t)), *leaves, use_reentrant=False), leaves, create_graph=True)
    for got in (moved, again, plain):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    with pytest.raises(RuntimeError, match="second derivatives"):
        moved[0].float().square().sum().backward()
    y = total(*outputs(how, *leaves))
    y.backward(create_graph=True)  # into .grad, and a second pass on top of it
    total(*outputs(how, *leaves)).backward()
    for t, b in zip(leaves, want):
        assert torch.equal(t.grad, 2 * b)
        t.grad = None
