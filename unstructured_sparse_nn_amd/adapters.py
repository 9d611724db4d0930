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

from . import binding as _b

_TYPES = {torch.float32: _b.F32, torch.bfloat16: _b.BF16}


def _rows(x, name, T, n, like, must=False):
    """x as a T x n matrix with contiguous rows, and its row stride."""
    if x.dtype is not like.dtype or x.device != like.device:
        raise TypeError(f"{name}: expected {like.dtype} on {like.device}, "
                        f"got {x.dtype} on {x.device}")
    if x.dim() != 2 or x.shape[0] != T or x.shape[1] != n:
        raise ValueError(f"{name}: expected shape ({T}, {n}), got {tuple(x.shape)}")
    ld, inner = x.stride()
    if (inner != 1 and n > 1) or (ld < n and T > 1):
        if must:
            raise ValueError(f"{name}: rows must be contiguous and must not overlap")
        x = x.contiguous()
        ld = n
    return x, ld if T > 1 else n


def _bank(x, ids, A, B, scale, ranks, T):
    """The argument struct of the adapters, after checks."""
    if A.dim() != 3 or B.dim() != 3 or A.shape[:2] != B.shape[:2]:
        raise ValueError(f"A (L, R, K) and B (L, R, M) expected, got {tuple(A.shape)} and "
                         f"{tuple(B.shape)}")
    L, R, K = A.shape
    if x.dtype not in _TYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if not x.is_cuda:
        raise TypeError("the adapters run on the GPU only")
    if A.dtype is not x.dtype or B.dtype is not x.dtype or A.device != x.device \
            or B.device != x.device:
        raise TypeError("A and B must have the activations' dtype and device")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous")
    if ids.dtype is not torch.int32 or ids.device != x.device or ids.dim() != 1 \
            or ids.shape[0] != T or not ids.is_contiguous():
        raise ValueError(f"ids: expected a contiguous int32 tensor of {T} on {x.device}")
    if scale is not None and (scale.dtype is not torch.float32 or scale.numel() != L
                              or scale.device != x.device or not scale.is_contiguous()):
        raise ValueError(f"scale: expected {L} contiguous float32 on {x.device}")
    if ranks is not None and (ranks.dtype is not torch.int32 or ranks.numel() != L
                              or ranks.device != x.device or not ranks.is_contiguous()):
        raise ValueError(f"ranks: expected {L} contiguous int32 on {x.device}")
    return _b.snack_lora(A, B, B.shape[2], K, L, R, scale, ranks)


def _check_t(t, T, R, like):
    if t.dtype is not torch.float32 or t.shape != (T, R) or not t.is_contiguous() \
            or t.device != like.device:
        raise ValueError(f"t: expected a contiguous float32 ({T}, {R}) tensor on {like.device}")


def lora_fwd(x, ids, A, B, scale=None, ranks=None, base=None, out=None, t=None):
    """``base + scale[a] * (x @ A[a].T) @ B[a]`` row by row, ``a = ids[row]``.

    x (T, K); base (T, M) or None; out (T, M), may be base; t (T, R) float32
    receives ``x @ A[a].T`` for :func:`lora_bwd`.  Rows of x, base and out may
    be strided."""
    if x.dim() != 2:
        raise ValueError(f"x: expected a matrix, got {tuple(x.shape)}")
    T = x.shape[0]
    bank = _bank(x, ids, A, B, scale, ranks, T)
    M = bank.M
    x, ldx = _rows(x, "x", T, bank.K, x)
    ldb = M
    if out is None:
        out = torch.empty(T, M, dtype=x.dtype, device=x.device)
        ldy = M
    else:
        _, ldy = _rows(out, "out", T, M, x, must=True)
    if base is not None:
        base, ldb = _rows(base, "base", T, M, x)
    if t is not None:
        _check_t(t, T, bank.R, x)
    dt = _TYPES[x.dtype]
    n = _b.snack_lora_workspace(bank, dt, T)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _b.snack_lora_fwd(bank, ids, T, x, ldx, base, ldb, out, ldy, t, ws, ws_bytes=n, dtype=dt)
    return out


def lora_bwd(dy, x, ids, A, B, scale=None, ranks=None, t=None, base=None, out=None,
             want=(True, True, True)):
    """Gradients (dx, dA, dB) of :func:`lora_fwd` from dy (T, M).

    t: what the forward stored (computed again without it).  base (T, K): the
    shared projection's input gradient, added to dx.  out (T, K) receives dx
    and may be base.  want: which of the three to compute (None for others)."""
    if x.dim() != 2:
        raise ValueError(f"x: expected a matrix, got {tuple(x.shape)}")
    T = x.shape[0]
    bank = _bank(x, ids, A, B, scale, ranks, T)
    K, M = bank.K, bank.M
    x, ldx = _rows(x, "x", T, K, x)
    dy, lddy = _rows(dy, "dy", T, M, x)
    if t is not None:
        _check_t(t, T, bank.R, x)
    dx, lddx, ldb = None, K, K
    if want[0]:
        if out is None:
            dx = torch.empty(T, K, dtype=x.dtype, device=x.device)
        else:
            dx = out
            _, lddx = _rows(out, "out", T, K, x, must=True)
        if base is not None:
            base, ldb = _rows(base, "base", T, K, x)
    else:
        base = None
    dA = torch.empty_like(A) if want[1] else None
    dB = torch.empty_like(B) if want[2] else None
    dt = _TYPES[x.dtype]
    n = _b.snack_lora_workspace(bank, dt, T, True)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _b.snack_lora_bwd(bank, ids, t, T, x, ldx, dy, lddy, base, ldb, dx, lddx, dA, dB, ws,
                      ws_bytes=n, dtype=dt)
    return dx, dA, dB


class _LoraFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, A, B, base, ids, scale, ranks):
        t = torch.empty(x.shape[0], A.shape[1], device=x.device)
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


class LoraAdapters(torch.nn.Module):
    """L trainable low-rank adapters of one projection.

    A starts normal with standard deviation 1/sqrt(in_features), B at zero, so
    an untrained adapter changes nothing.  ``ranks`` (a list) may give each
    adapter its own rank up to ``rank``; ``alpha / rank`` is the scale."""

    def __init__(self, in_features: int, out_features: int, adapters: int, rank: int,
                 alpha: float = 16.0, ranks=None, dtype=torch.float32, device="cuda"):
        super().__init__()
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

    def forward(self, x, ids, base=None):
        """base + each row's adapter applied to x (rows of x: tokens)."""
        if torch.is_grad_enabled():
            return _LoraFn.apply(x, self.A, self.B, base, ids, self.scale, self.ranks)
        return lora_fwd(x, ids, self.A, self.B, self.scale, self.ranks, base)
