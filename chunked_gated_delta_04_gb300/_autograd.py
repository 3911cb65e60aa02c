"""What the package's autograd functions share."""
from __future__ import annotations

import functools

import torch


class _NoSecondDerivative(torch.autograd.Function):
    """Hands the first n tensors on as results of all the others, and refuses to be differentiated."""

    @staticmethod
    def forward(ctx, name, n, *tensors):
        ctx.name, ctx.count = name, len(tensors)
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no second derivative: its gradients cannot be differentiated")


def first_order(name):
    """Decorates a Function's backward that computes its gradients outside autograd.  With create_graph they
    would count as constants, and a second derivative would lack every term through them.  Here they
    depend on the saved tensors and the incoming gradients through a node that refuses.  (torch's once_differentiable
    hangs its refusal on no input: autograd.grad, which walks only towards the inputs that it is asked for, passes it by,
    and gradients that come in as constants, as those of a sum, leave it out.)"""
    def decorate(backward):
        @functools.wraps(backward)
        def run(ctx, *grads):
            with torch.no_grad():
                outs = backward(ctx, *grads)
            if not torch.is_grad_enabled():
                return outs
            given = [t for t in outs if t is not None]
            sources = [t for t in (*ctx.saved_tensors, *grads) if t is not None]
            handed = iter(_NoSecondDerivative.apply(name, len(given), *[t.detach() for t in given], *sources))
            return tuple(None if t is None else next(handed) for t in outs)

        return run

    return decorate


def link(state):
    """Nothing of a state, connected to it: what a Function saves of a state that it does not need, so that its
    gradients depend on it (see first_order) while its owner may change it in place."""
    return state[:0].clone() if state is not None and state.requires_grad else None
