"""Torch-facing calls of dropout (``snack_dropout``): the mask comes from a
counter-based generator and is never stored.

Element i of a call is dropped or kept by ``seed``, ``step`` and i alone, so the
backward pass (and a recomputed forward, given the same step) finds the same mask
again.  One seed to a place in the model and one step to a call give independent
masks.  ``step`` may be a number or one int64 on the GPU, which is read when the
kernel runs: a captured graph whose step is counted up between replays draws anew.

The modules count their calls in training where a call names no step
(:class:`CountedSteps`).
"""
from __future__ import annotations

import copy
import random
import threading
import weakref
from collections import OrderedDict

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


# Calls of a module that may still be run again.
RECENT = 4096
_in_backward = torch._C._current_graph_task_id  # -1: not
_local = threading.local()
_known = weakref.WeakKeyDictionary()  # module: [its step after the last call, {draw: step}]


def _draw() -> int:
    """63 bits of torch's generator of the CPU, in half the time of a new tensor's."""
    number = getattr(_local, "number", None)
    if number is None:
        with torch.inference_mode(False):
            number = _local.number = torch.empty((), dtype=torch.int64, device="cpu")
    return number.random_().item()


class CountedSteps:
    """The steps of a module's calls: ``self.step``, counted up.

    A call that is run again (``torch.utils.checkpoint``, either form) takes the
    step of its first run.  It is known by a number that every call draws from
    torch's generator of the CPU, whose state a recomputation restores: as of
    torch's own dropout, calls from one state of the generator drop the same
    elements, unless ``self.step`` was set between them.  A call that the backward
    runs from another state (``preserve_rng_state=False``), or again after RECENT
    others, is refused, and so is a counted step in a capture: every replay would
    drop the same elements.

    A deep copy has a seed of its own, made from this one's and the number of copies
    made before: layers that are copies of one draw independent masks."""

    copies = 0

    def __deepcopy__(self, memo):
        make, args, state = self.__reduce_ex__(2)[:3]
        other = memo[id(self)] = make(*args)
        other.__setstate__(copy.deepcopy(state, memo))
        if self.seed is not None:
            other.seed = random.Random(f"{self.seed} {self.copies}").getrandbits(62)
        other.copies = 0
        self.copies += 1
        return other

    def _next_step(self, x):
        if x.is_cuda and torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"{type(self).__name__}: a captured call has to name its step, one "
                               "int64 on the GPU that is counted up between the replays")
        draw = _draw()
        in_backward = _in_backward() != -1
        known = _known.get(self)
        if known is None or (known[0] != self.step and not in_backward):
            known = _known[self] = [self.step, OrderedDict()]
        step = known[1].get(draw)
        if step is None:
            if in_backward:
                raise RuntimeError(f"{type(self).__name__}: a call that the backward runs again "
                                   "has no known step; name the step, or let the recomputation "
                                   "restore torch's generator of the CPU")
            if len(known[1]) >= RECENT:
                known[1].popitem(last=False)
            step = known[1][draw] = self.step
            self.step = known[0] = step + 1
        return step


class Dropout(CountedSteps, torch.nn.Module):
    """Dropout in training, with a residual added in the same pass if given.

    ``step`` counts the calls in training (no part of the state dict; a call that
    activation checkpointing runs again counts once, :class:`CountedSteps`); a call
    may name its own, a number or one int64 on the GPU.  A captured call has to:
    with the latter, counted up between replays, each draws anew."""

    def __init__(self, p: float, seed: int | None = None):
        super().__init__()
        if not 0 <= p <= 1:
            raise ValueError("p: from 0 to 1")
        self.p, self.seed, self.step = p, random_seed() if seed is None else seed, 0

    def forward(self, x, residual=None, step=None):
        if not self.training or self.p == 0:
            return x if residual is None else residual + x
        if step is None:
            step = self._next_step(x)
        return _DropoutFn.apply(x, residual, self.p, self.seed, step)

    def extra_repr(self):
        return f"p={self.p}"
