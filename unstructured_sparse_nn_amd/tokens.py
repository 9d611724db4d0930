"""Torch-facing calls of the two ends of a model (``snack_embed_*``,
``snack_logp_*``): rows looked up by token, with the table's gradient, and the
log-probabilities of target tokens from logits, with the logits' gradient.

Token numbers are int32 or int64 of any shape.  A negative one means no token
(a row of zeros, log-probability 0, no gradient); one past the table gives NaN
and no gradient of the table.
"""
from __future__ import annotations

import torch

from .native import calls


def embed_fwd(ids, weight, scale: float = 1.0, out=None):
    """``scale * weight[ids]``, weight (V, D); out of the shape ids + (D,) counts
    as changed in place.  Autograd does not record this call
    (:class:`TokenEmbedding` does)."""
    return calls().embed_fwd(ids, weight, scale, out)


def embed_bwd(dy, ids, rows: int, scale: float = 1.0, base=None, out=None):
    """The gradient (rows, D) of the table of :func:`embed_fwd` from dy.

    base: a gradient that is there already (of a head that shares the table, of
    the steps before), added in the same pass; out may be base (an out that shares
    other memory is refused) and counts as changed in place."""
    return calls().embed_bwd(dy, ids, rows, scale, base, out)


class _EmbedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = weight.shape[0], scale
        return embed_fwd(ids, weight, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        return embed_bwd(gy, ctx.saved_tensors[0], ctx.rows, ctx.scale), None, None


class TokenEmbedding(torch.nn.Module):
    """A trainable table of ``rows`` tokens by ``features``, looked up and scaled.
    Starts normal with standard deviation 0.02.

    Forward and backward can be captured into a graph; as with any torch module,
    no output of an eager step may still hold this parameter's autograd graph
    while the backward is captured."""

    def __init__(self, rows: int, features: int, scale: float = 1.0, dtype=torch.float32,
                 device="cuda"):
        super().__init__()
        self.scale = scale
        self.weight = torch.nn.Parameter(
            torch.randn(rows, features, device=device).mul_(0.02).to(dtype))

    def forward(self, ids):
        return _EmbedFn.apply(self.weight, ids, self.scale)

    def extra_repr(self):
        return f"{self.weight.shape[0]}, {self.weight.shape[1]}, scale={self.scale}"


def logp_fwd(logits, targets):
    """(logp, norm): the log-probability of each row's target (float32), and the
    row's largest logit with the logarithm of the sum of exp(logit - largest),
    one axis of 2 more, for :func:`logp_bwd`.  Their sum is the log of the
    partition function.  Rows are read where they lie if they are evenly apart;
    others are copied first, as those of ``logits[:, :-1]`` of several sequences are,
    here and in the backward (all rows with -1 as the last target are not).
    Autograd does not record this call (:func:`token_logps` does)."""
    return calls().logp_fwd(logits, targets)


def logp_bwd(dlogp, logits, targets, norm, out=None):
    """The gradient of :func:`logp_fwd`'s logp by the logits.

    out may be the logits themselves (another out that shares memory is refused)
    and counts as changed in place.  Rows whose dlogp is 0 are zeros and are not
    read."""
    return calls().logp_bwd(dlogp, logits, targets, norm, out)


class _LogpFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets):
        logp, norm = logp_fwd(logits, targets)
        ctx.save_for_backward(logits, targets, norm)
        return logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        return logp_bwd(g, *ctx.saved_tensors), None


def token_logps(logits, targets):
    """The log-probability of each target under its row of logits: float32 of the
    targets' shape, 0 where a target is negative.  For the next token of each,
    ``targets = ids.roll(-1, 1)`` with its last column -1 needs no copy of the logits
    (:func:`logp_fwd`)."""
    return _LogpFn.apply(logits, targets)
