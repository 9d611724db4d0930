"""Torch-facing calls of gradient clipping (``snack_grad_*``): the 2-norm over
many gradients and their scaling, in two launches per 112 tensors.

The list of tensors is read anew by every call; nothing is kept between calls
and nothing waits for the GPU.
"""
from __future__ import annotations

import torch

from .native import calls


def grad_norm(grads):
    """sqrt of the sum of squares over all elements of all tensors, a float32
    scalar on their device (float32 and bfloat16 tensors, mixed as they come)."""
    grads = list(grads)
    if not grads:
        return torch.zeros(())
    return calls().clip(grads, None, None, 0.0)


def clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None):
    """Scale the tensors by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (tensors of the same shapes); returns the norm before scaling.
    Refused where an output shares memory with another output or with another
    gradient (one gradient twice, in place, too).
    A NaN norm makes every output NaN; an infinite one zeroes the finite ones."""
    grads = list(grads)
    outs = None if out is None else list(out)
    if not grads:
        if outs:
            raise ValueError(f"0 gradients but {len(outs)} outputs")
        return torch.zeros(())
    return calls().clip(grads, outs, max_norm, eps)


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6):
    """:func:`clip_grads` on the ``.grad`` of the parameters that have one; each
    parameter once."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    return clip_grads([p.grad for p in parameters if p.grad is not None], max_norm, eps)
