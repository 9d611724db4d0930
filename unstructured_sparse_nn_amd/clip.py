"""Torch-facing calls of gradient clipping (``snack_grad_*``): the 2-norm over
many gradients and their scaling, in two launches per 112 tensors.

The list of tensors is read anew by every call; nothing is kept between calls
and nothing waits for the GPU.
"""
from __future__ import annotations

import torch
from torch._prims_common import is_non_overlapping_and_dense

from . import binding as _b


def _check(grads, outs):
    dev = grads[0].device
    if dev.type != "cuda":
        raise TypeError("gradients must be on the GPU")
    for g in grads:
        if g.device != dev:
            raise TypeError("gradients must be on one device")
        if not g.is_contiguous() and not is_non_overlapping_and_dense(g):
            raise ValueError("a gradient must fill its memory without gaps or overlaps")
    if outs is None:
        return
    if len(outs) != len(grads):
        raise ValueError(f"{len(grads)} gradients but {len(outs)} outputs")
    for g, o in zip(grads, outs):
        if o.shape != g.shape or o.dtype is not g.dtype or o.device != dev:
            raise ValueError("an output must have its gradient's shape, dtype and device")
        if not (g.is_contiguous() and o.is_contiguous()) and o.stride() != g.stride():
            raise ValueError("an output must have its gradient's strides")


def grad_norm(grads):
    """sqrt of the sum of squares over all elements of all tensors, a float32
    scalar on their device (float32 and bfloat16 tensors, mixed as they come)."""
    grads = list(grads)
    if not grads:
        return torch.zeros(())
    _check(grads, None)
    dev = grads[0].device
    norm = torch.empty((), device=dev)
    n = _b.snack_grad_workspace(len(grads))
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _b.snack_grad_norm(_b.snack_grad_table(grads), len(grads), norm, ws, ws_bytes=n)
    return norm


def clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None):
    """Scale the tensors by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (tensors of the same shapes); returns the norm before scaling.
    A NaN norm makes every output NaN; an infinite one zeroes the finite ones."""
    grads = list(grads)
    outs = None if out is None else list(out)
    if not grads:
        if outs:
            raise ValueError(f"0 gradients but {len(outs)} outputs")
        return torch.zeros(())
    _check(grads, outs)
    dev = grads[0].device
    norm = torch.empty((), device=dev)
    n = _b.snack_grad_workspace(len(grads))
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _b.snack_grad_clip(_b.snack_grad_table(grads, outs), len(grads), max_norm, eps, norm, ws,
                       ws_bytes=n)
    torch.autograd.graph.increment_version(grads if outs is None else outs)
    return norm


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6):
    """:func:`clip_grads` on the ``.grad`` of the parameters that have one."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    return clip_grads([p.grad for p in parameters if p.grad is not None], max_norm, eps)
