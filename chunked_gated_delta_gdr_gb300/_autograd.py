"""What the backwards of the differentiable functions share."""
from __future__ import annotations

import torch


class _FirstOnly(torch.autograd.Function):
    """Gradients as they are, with the inputs that they depend on but no derivative."""

    @staticmethod
    def forward(ctx, name, grads, *inputs):
        ctx.name = name
        return tuple(grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has first derivatives only: its gradients cannot be "
                           "differentiated")


def first_only(name, grads, *inputs):
    """A backward's gradients, computed by kernels from ``inputs``.  Where autograd records the
    backward itself (``create_graph=True``), differentiating them is an error; without this they
    would count as constants, without a word."""
    if torch.is_grad_enabled():
        inputs = [t for t in inputs if t is not None and t.requires_grad]
        if inputs:
            return _FirstOnly.apply(name, grads, *inputs)
    return grads
