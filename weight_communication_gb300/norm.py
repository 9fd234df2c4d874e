"""Root-mean-square norm of a residual stream, whose input is kept in 8 bits for
the backward pass.

    forward:  t = x + add (or x),  r = 1 / sqrt(mean of t^2 + eps),  y = t * r * weight
    backward: n = t^ * r,
              dx = r * (dy * weight - n * mean of (dy * weight * n)) + add
              dweight = sum over the rows of dy * n

where t^ is what the kept codes stand for (e4m3 with one fp32 scale per 128
values of a row, as `fp8.quantize` makes them), and the backward pass's add is the
gradient that reaches t past the norm.  Sums are in fp32, the same bits every run.

    y, total, kept = norm.rms(x, weight, add=residual, save=True)
    dx, dweight = norm.rms_grad(dy, weight, kept, add=dtotal)   # dx: of x and of residual
"""
from __future__ import annotations

import torch

from . import binding
from .fp8 import Fp8Tensor


class Kept:
    """What a forward pass keeps: t as an Fp8Tensor [rows, columns] and r, fp32 [rows]."""

    __slots__ = ("input", "rstd")

    def __init__(self, input: Fp8Tensor, rstd: torch.Tensor):
        self.input, self.rstd = input, rstd


def rms(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, add: torch.Tensor | None = None,
        save: bool = False, stream=None):
    """(y, t), or with save (y, t, Kept); t is x + add rounded to x's type, x itself
    without add.  x, add: float32 or bfloat16, matrices whose rows are consecutive
    values, or contiguous tensors [.., columns], of up to 16384 columns; weight
    [columns] in either type."""
    y, total, rstd, parts = binding.on_stream(stream, x.device, binding.calls().rms_norm, x, weight, eps, add, save)
    total = x if total is None else total
    return (y, total, Kept(Fp8Tensor._made(parts), rstd)) if save else (y, total)


def rms_grad(dy: torch.Tensor, weight: torch.Tensor, kept: Kept, add: torch.Tensor | None = None,
             dweight: torch.Tensor | None = None, accumulate: bool = False, stream=None):
    """(dx, dweight): dx of dy's shape and type, dweight fp32 [columns] or the
    given buffer (either type), written or, with accumulate, added to."""
    return binding.on_stream(stream, dy.device, binding.calls().rms_norm_grad, dy, weight, kept.rstd,
                             kept.input._parts, add, dweight, accumulate)
