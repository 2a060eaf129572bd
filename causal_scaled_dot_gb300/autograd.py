"""What the library's autograd functions have in common: gradients that cannot be differentiated again say so."""
from __future__ import annotations

import torch


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
