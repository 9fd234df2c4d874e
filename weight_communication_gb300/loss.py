"""Softmax cross entropy of a linear output layer over a large vocabulary, in
pieces of the vocabulary and without keeping the logits.

    s = x weight^T,  lse[t] = log sum over v of exp(s[t][v])
    loss[t] = lse[t] - s[t][targets[t]]
    d[t][v] = dlosses[t] * (exp(s[t][v] - lse[t]) - [v = targets[t]])
    dx = d weight,  dw = d^T x

x [.., D] and weight [V, D] are bf16 and multiplied on the tensor cores with fp32
sums.  A target outside [0, V) is padding: its loss is 0, and nothing in its row of
x reaches a gradient.  The backward pass multiplies the logits again, the same bits, a
piece of the vocabulary at a time, with d rounded to bf16 for the products (not for up to
four tokens of up to 4096 values).  lse is one fp32 number, so each exponential of d carries
its rounding, |lse| 2^-24 of itself.  The same bits every run.

    losses, lse = loss.cross_entropy(x, weight, targets, save=True)
    dx, dw = loss.cross_entropy_grad(x, weight, targets, lse, 1.0 / tokens)
"""
from __future__ import annotations

import torch

from . import binding


def cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, save: bool = False,
                  stream=None):
    """Each token's loss, fp32 of targets' shape; with save, (losses, lse).
    targets: int32 or int64, contiguous, one for each row of x."""
    losses, lse = binding.on_stream(stream, x.device, binding.calls().cross_entropy, x, weight, targets)
    return (losses, lse) if save else losses


def cross_entropy_grad(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                       dlosses: float | torch.Tensor, dw: torch.Tensor | None = None,
                       dw_dtype: torch.dtype | None = None, accumulate: bool = False,
                       needs_dx: bool = True, needs_dw: bool = True, stream=None):
    """(dx, dw): dx bf16 of x's shape; dw [V, D], a new tensor of dw_dtype (bf16
    unless given), or the given buffer (bf16 or fp32, rows that start anywhere),
    written or, with accumulate, added to, which shares no memory with the inputs (a
    weight cannot be updated in place).  dlosses: the gradient of each token's
    loss, fp32 [tokens], or one Python number for all.  A gradient that is not needed is
    not computed, and None."""
    return binding.on_stream(stream, x.device, binding.calls().cross_entropy_grad, x, weight, targets, lse,
                             dlosses, needs_dx, needs_dw, dw, dw_dtype, accumulate)
