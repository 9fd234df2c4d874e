"""Embedding lookup with scaling, and the gradient of its table.

    lookup: out[t] = scale * table[ids[t] - first_row]
    grad:   dtable[v] = scale * sum of dy[t] over the t with ids[t] - first_row = v

The table may be all of a vocabulary or the rows [first_row, first_row + V) of
one that is split over ranks: ids outside read as zero and receive nothing, so
the ranks' lookups add up to the whole one, and negative ids are padding.
The gradient is a deterministic sum (the same bits every run), which keeps
data-parallel replicas equal, and can be added to the gradient of earlier
micro-batches.
"""
from __future__ import annotations

import torch

from . import binding


def lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, first_row: int = 0,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[*ids.shape, D] of the table's type (float32 or bfloat16); ids int32 or
    int64, contiguous, of any shape.  `out`: a matrix [ids.numel(), D] to write instead of a
    new tensor (its rows may be further apart than D)."""
    return binding.on_stream(stream, table.device, binding.calls().embedding, table, ids, scale,
                             first_row, out)


def grad(dy: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0, first_row: int = 0,
         out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
         accumulate: bool = False, stream=None) -> torch.Tensor:
    """The table's gradient [rows, D] from dy [*ids.shape, D]: a new tensor of
    out_dtype (dy's type by default), or written to `out`; with accumulate,
    added to what `out` holds (rows without a token are left alone)."""
    return binding.on_stream(stream, dy.device, binding.calls().embedding_grad, dy, ids, rows, scale,
                             first_row, out, out_dtype, accumulate)
