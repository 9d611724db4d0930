"""Torch-facing calls of the low-rank adapters (``snack_lora_*``): many
adapters beside one shared projection, each token using its own.

Factors are stored by rank: ``A`` (L, R, K) and ``B`` (L, R, M), so adapter l
adds ``scale[l] * B[l].T @ A[l]`` to a weight of M x K.  ``ids`` (int32) names
the adapter of each token; a negative id means none.  Nothing here waits for
the GPU; buffers come from torch and every kernel runs on torch's current
stream.
"""
from __future__ import annotations

import torch

from .dropout import CountedSteps, dropout_bwd, dropout_fwd, random_seed
from .native import calls


def lora_fwd(x, ids, A, B, scale=None, ranks=None, base=None, out=None, t=None):
    """``base + scale[a] * (x @ A[a].T) @ B[a]`` row by row, ``a = ids[row]``.

    x (T, K); base (T, M) or None; out (T, M), may be base; t (T, R) float32
    receives ``x @ A[a].T`` for :func:`lora_bwd`.  Rows of x, base and out may
    be strided.  An out or t that shares memory with anything else is refused.
    Autograd does not record this call (:class:`LoraAdapters` does); out and t
    count as changed in place."""
    return calls().lora_fwd(x, ids, A, B, scale, ranks, base, out, t)


def lora_bwd(dy, x, ids, A, B, scale=None, ranks=None, t=None, base=None, out=None,
             want=(True, True, True)):
    """Gradients (dx, dA, dB) of :func:`lora_fwd` from dy (T, M).

    t: what the forward stored (computed again without it).  base (T, K): the
    shared projection's input gradient, added to dx.  out (T, K) receives dx, may
    be base (an out that shares memory with anything else is refused) and counts
    as changed in place.  want: which of the three to compute (None for others).
    Autograd does not record this call."""
    return calls().lora_bwd(dy, x, ids, A, B, scale, ranks, t, base, out, *want)


class _LoraFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, A, B, base, ids, scale, ranks):
        t = torch.empty(x.shape[0], A.shape[1], dtype=torch.float32, device=x.device)
        y = lora_fwd(x, ids, A, B, scale, ranks, base, t=t)
        ctx.save_for_backward(x, A, B, ids, scale, ranks, t)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, A, B, ids, scale, ranks, t = ctx.saved_tensors
        want = ctx.needs_input_grad[:3]
        dx = dA = dB = None
        if any(want):
            dx, dA, dB = lora_bwd(gy, x, ids, A, B, scale, ranks, t, want=want)
        return dx, dA, dB, gy if ctx.needs_input_grad[3] else None, None, None, None


class _DroppedLoraFn(torch.autograd.Function):
    """The same on dropout(x), which the backward makes again from x."""

    @staticmethod
    def forward(ctx, x, A, B, base, ids, scale, ranks, p, seed, step):
        on_gpu = isinstance(step, torch.Tensor)
        t = torch.empty(x.shape[0], A.shape[1], dtype=torch.float32, device=x.device)
        y = lora_fwd(dropout_fwd(x, p, seed, step), ids, A, B, scale, ranks, base, t=t)
        ctx.save_for_backward(x, A, B, ids, scale, ranks, t, step if on_gpu else None)
        ctx.args = p, seed, None if on_gpu else step
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        x, A, B, ids, scale, ranks, t, step = ctx.saved_tensors
        p, seed, number = ctx.args
        step = number if step is None else step
        want = ctx.needs_input_grad[:3]
        dx = dA = dB = None
        if any(want):
            if want[1]:
                x = dropout_fwd(x, p, seed, step)
            dx, dA, dB = lora_bwd(gy, x, ids, A, B, scale, ranks, t, want=want)
            if want[0]:
                dx = dropout_bwd(dx, p, seed, step, out=dx)
        return (dx, dA, dB, gy if ctx.needs_input_grad[3] else None, *[None] * 6)


class LoraAdapters(CountedSteps, torch.nn.Module):
    """L trainable low-rank adapters of one projection.

    A starts normal with standard deviation 1/sqrt(in_features), B at zero, so
    an untrained adapter changes nothing.  ``ranks`` (a list) may give each
    adapter its own rank up to ``rank``; ``alpha / rank`` is the scale.

    ``dropout``: in training, the adapters see x with that share of its elements
    dropped (base does not).  Its mask comes from ``seed`` (drawn from torch's
    generator if None) and ``step``, which counts the calls in training (one that
    activation checkpointing runs again once) and is no part of the state dict; a
    call may name its own, a number or one int64 on the GPU (:mod:`.dropout`).

    Forward and backward can be captured into a graph; with dropout the captured
    call has to name its step, on the GPU if replays are to draw anew.  As with
    any torch module, no output of an eager step may still hold these parameters'
    autograd graph while the backward is captured: torch would join the eager
    stream to the capture and end the process."""

    dropout, seed, step = 0.0, None, 0  # of modules that were pickled without them

    def __init__(self, in_features: int, out_features: int, adapters: int, rank: int,
                 alpha: float = 16.0, ranks=None, dtype=torch.float32, device="cuda",
                 dropout: float = 0.0, seed: int | None = None):
        super().__init__()
        if not 0 <= dropout <= 1:
            raise ValueError("dropout: from 0 to 1")
        if ranks is not None and (len(ranks) != adapters
                                  or not all(0 < r <= rank for r in ranks)):
            raise ValueError("ranks: one per adapter, from 1 to rank")
        self.A = torch.nn.Parameter(torch.randn(adapters, rank, in_features, device=device)
                                    .mul_(in_features ** -0.5).to(dtype))
        self.B = torch.nn.Parameter(torch.zeros(adapters, rank, out_features, dtype=dtype,
                                                device=device))
        of = ranks if ranks is not None else [rank] * adapters
        self.register_buffer("scale", torch.tensor([alpha / r for r in of], dtype=torch.float32,
                                                   device=device))
        self.register_buffer("ranks", None if ranks is None else torch.tensor(
            ranks, dtype=torch.int32, device=device))
        self.dropout, self.seed, self.step = dropout, seed, 0
        if dropout > 0 and seed is None:
            self.seed = random_seed()

    def _apply(self, fn, recurse=True):
        # the kernels read scale as float32 and ranks as int32, whatever type the
        # module is cast to: casts move the buffers to another device only
        kept = {k: v for k, v in self._buffers.items() if v is not None}
        super()._apply(fn, recurse)
        for k, v in kept.items():
            if self._buffers[k].dtype != v.dtype:
                self._buffers[k] = v.to(self._buffers[k].device)
        return self

    def forward(self, x, ids, base=None, step=None):
        """base + each row's adapter applied to x (rows of x: tokens)."""
        if self.training and self.dropout > 0:
            if step is None:
                step = self._next_step(x)
            return _DroppedLoraFn.apply(x, self.A, self.B, base, ids, self.scale, self.ranks,
                                        self.dropout, self.seed, step)
        if torch.is_grad_enabled():
            return _LoraFn.apply(x, self.A, self.B, base, ids, self.scale, self.ranks)
        return lora_fwd(x, ids, self.A, self.B, self.scale, self.ranks, base)
