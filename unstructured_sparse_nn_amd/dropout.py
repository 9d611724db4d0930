"""Torch-facing calls of dropout (``snack_dropout``): the mask comes from a
counter-based generator and is never stored.

Element i of a call is dropped or kept by ``seed``, ``step`` and i alone, so the
backward pass (and a recomputed forward) finds the same mask again.  One seed to
a place in the model and one step to a call give independent masks.  ``step``
may be a number or one int64 on the GPU, which is read when the kernel runs: a
captured graph whose step is counted up between replays draws anew.
"""
from __future__ import annotations

import torch

from .native import calls


def _apply(x, p, seed, step, residual, out):
    on_gpu = isinstance(step, torch.Tensor)
    return calls().dropout(x, p, seed, 0 if on_gpu else step, step if on_gpu else None, residual,
                           out)


def dropout_fwd(x, p: float, seed: int, step=0, residual=None, out=None):
    """``residual + x * mask / (1 - p)``; p counts in steps of 2^-16.

    x and residual float32 or bfloat16 of one shape; out may be either of them
    and counts as changed in place.  Autograd does not record this call
    (:class:`Dropout` does)."""
    return _apply(x, p, seed, step, residual, out)


def dropout_bwd(dy, p: float, seed: int, step=0, out=None):
    """The gradient of :func:`dropout_fwd` by x (by the residual it is dy)."""
    return _apply(dy, p, seed, step, None, out)


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, step):
        on_gpu = isinstance(step, torch.Tensor)
        ctx.save_for_backward(step if on_gpu else None)
        ctx.args = p, seed, None if on_gpu else step
        return dropout_fwd(x, p, seed, step, residual)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        p, seed, step = ctx.args
        step = ctx.saved_tensors[0] if step is None else step
        dx = dropout_bwd(gy, p, seed, step) if ctx.needs_input_grad[0] else None
        return dx, gy if ctx.needs_input_grad[1] else None, None, None, None


def random_seed() -> int:
    """A seed from torch's generator of the CPU, whatever the default device."""
    return int(torch.randint(0, 2 ** 62, (), device="cpu"))


class Dropout(torch.nn.Module):
    """Dropout in training, with a residual added in the same pass if given.

    ``step`` counts the calls in training (no part of the state dict); a call may
    name its own, a number or one int64 on the GPU."""

    def __init__(self, p: float, seed: int | None = None):
        super().__init__()
        if not 0 <= p <= 1:
            raise ValueError("p: from 0 to 1")
        self.p, self.seed, self.step = p, random_seed() if seed is None else seed, 0

    def forward(self, x, residual=None, step=None):
        if not self.training or self.p == 0:
            return x if residual is None else residual + x
        if step is None:
            step, self.step = self.step, self.step + 1
        return _DropoutFn.apply(x, residual, self.p, self.seed, step)

    def extra_repr(self):
        return f"p={self.p}"
