"""What the library's calls have in common towards autograd: gradients that cannot be differentiated again say so, and
forward-mode tangents, which no call carries on, are refused."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad


class _Tied(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gradient, *sources):
        return gradient.detach()  # not a view that may not be changed in place

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("second derivatives through this library's kernels are not available: what was differentiated with "
                           "create_graph=True depends on tensors that require a gradient")


def tied(gradient, *sources):
    """A gradient that a kernel made from `sources` in a backward pass that is itself recorded.  Where one of them requires
    a gradient so does the result, and asking for that raises; else it is a constant.  (once_differentiable looks at the
    upstream gradients alone: under a constant one, a gradient that depends on saved tensors would count as a constant.)"""
    if gradient is None or not any(s is not None and s.requires_grad for s in sources):
        return gradient
    return _Tied.apply(gradient, *(s for s in sources if s is not None))


def refuse_tangents(*tensors):
    """Raises where one of a call's inputs is a dual tensor: the result would come back without its tangent, as a constant."""
    # Outside of dual_level there are none; where torch does not tell (the name is not a documented one) each input is asked.
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("an input carries a forward-mode tangent, which this call does not: use reverse mode, or pass the primal")
