"""Torch-facing losses of answers by the log-probabilities of their tokens
(``snack_preference``, ``snack_policy_loss``).

Log-probabilities are float32, one a token.  ``starts`` (int32, one more than
sequences) says where each sequence begins among them; without it every row of
a matrix is a sequence.  ``mask`` (bool or uint8, the same shape) leaves tokens
out of every sum and count.  The losses are scalars on the GPU; nothing here
waits for it.  The backwards of :func:`preference_loss` and :func:`policy_loss`
compute the sums again; ``*_grads`` give loss and gradient of one call.
"""
from __future__ import annotations

import torch

from . import binding as b
from .native import calls

FORMS = {"sigmoid": b.PREF_SIGMOID, "hinge": b.PREF_HINGE, "squared": b.PREF_SQUARED}


def _one_of(value, choices, name):
    if value not in choices:
        raise ValueError(f"{name}: one of {', '.join(choices)}")
    return value


def preference_grads(logps, starts=None, ref=None, mask=None, beta: float = 0.1,
                     smoothing: float = 0.0, form: str = "sigmoid", average: bool = False,
                     dloss=None, want=(True, True)):
    """(loss, rewards, dlogps) of :func:`preference_loss` in one call.

    dloss: the gradient of the loss (one float32 on the GPU; 1 without it).  want:
    whether loss and rewards, and whether the gradient, are computed (None for
    what is not)."""
    return calls().preference(logps, starts, ref, mask, beta, smoothing,
                              FORMS[_one_of(form, FORMS, "form")], average, dloss, *want)


class _PreferenceFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logps, starts, ref, mask, args):
        ctx.save_for_backward(logps, starts, ref, mask)
        ctx.args = args
        loss, rewards, _ = preference_grads(logps, starts, ref, mask, *args, want=(True, False))
        ctx.mark_non_differentiable(rewards)
        return loss, rewards

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, _):
        return preference_grads(*ctx.saved_tensors, *ctx.args, dloss=g,
                                want=(False, True))[2], None, None, None, None


def preference_loss(logps, starts=None, ref=None, mask=None, beta: float = 0.1,
                    smoothing: float = 0.0, form: str = "sigmoid", average: bool = False):
    """The mean loss of pairs of sequences, 2p preferred to 2p + 1, and their
    rewards (pairs, 2).

    With h the difference of the two sums of ``logps - ref`` (``average``: means)
    and z = beta h: "sigmoid" ``-log sigmoid(z)`` (``smoothing`` of it with the pair
    turned round), "hinge" ``max(0, 1 - z)``, "squared" ``(h - 1 / (2 beta))^2``.  A
    reward is beta times its sequence's sum.  Gradients go to logps."""
    return _PreferenceFn.apply(logps, starts, ref, mask,
                               (beta, smoothing, _one_of(form, FORMS, "form"), average))


def policy_grads(logps, old, advantages, starts=None, ref=None, mask=None, clip=(0.2, 0.2),
                 kl: float = 0.0, average: str = "tokens", by: str = "sequences", dloss=None,
                 want=(True, True)):
    """(loss, stats, dlogps) of :func:`policy_loss` in one call; dloss and want as
    of :func:`preference_grads`."""
    low, high = clip
    return calls().policy(logps, old, advantages, starts, ref, mask, low, high, kl,
                          _one_of(by, ("tokens", "sequences"), "by") == "tokens",
                          _one_of(average, ("tokens", "sequences"), "average") == "sequences",
                          dloss, *want)


class _PolicyFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logps, old, advantages, starts, ref, mask, args):
        ctx.save_for_backward(logps, old, advantages, starts, ref, mask)
        ctx.args = args
        loss, stats, _ = policy_grads(logps, old, advantages, starts, ref, mask, *args,
                                      want=(True, False))
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g, _):
        return (policy_grads(*ctx.saved_tensors, *ctx.args, dloss=g, want=(False, True))[2],
                *[None] * 6)


def policy_loss(logps, old, advantages, starts=None, ref=None, mask=None, clip=(0.2, 0.2),
                kl: float = 0.0, average: str = "tokens", by: str = "sequences"):
    """The clipped policy loss with a KL term, and stats (2,): the mean over the
    tokens of the KL estimate, and of whether the clip decided.

    With r = exp(logps - old) (old None: r = 1) and A the advantage of the token
    (``by`` "tokens") or of its sequence, at each token
    ``-min(r A, clamp(r, 1 - clip[0], 1 + clip[1]) A) + kl (exp(k) - k - 1)``, k = ref - logps
    (ref None: no KL term; with kl 0 ref is for stats alone), averaged over all tokens,
    or (``average`` "sequences") over each sequence's and then over the sequences.
    Gradients go to logps."""
    return _PolicyFn.apply(logps, old, advantages, starts, ref, mask,
                           (clip, kl, _one_of(average, ("tokens", "sequences"), "average"),
                            _one_of(by, ("tokens", "sequences"), "by")))
