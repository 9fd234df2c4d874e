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


def _flat(ids: torch.Tensor) -> torch.Tensor:
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids if ids.dim() == 1 else ids.view(-1)


def lookup(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, first_row: int = 0,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """[*ids.shape, D] of the table's type (float32 or bfloat16); ids int32 or
    int64 of any shape.  `out`: a matrix [ids.numel(), D] to write instead of a
    new tensor (its rows may be further apart than D)."""
    flat = _flat(ids)
    if table.dim() != 2:
        raise ValueError(f"table must be a matrix, got shape {tuple(table.shape)}")
    given = out
    if out is None:
        with binding.allocating_on(stream):
            out = torch.empty((flat.numel(), table.shape[1]), dtype=table.dtype, device=table.device)
    binding.embedding(table, flat, out, scale, first_row, stream)
    return out.view(*ids.shape, table.shape[1]) if given is None and ids.dim() != 1 else out


def grad(dy: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0, first_row: int = 0,
         out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
         accumulate: bool = False, stream=None) -> torch.Tensor:
    """The table's gradient [rows, D] from dy [*ids.shape, D]: a new tensor of
    out_dtype (dy's type by default), or written to `out`; with accumulate,
    added to what `out` holds (rows without a token are left alone)."""
    flat = _flat(ids)
    D = dy.shape[-1]
    if dy.dim() != 2:
        if dy.shape[:-1] != ids.shape or not dy.is_contiguous():
            raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*ids.shape, D)}, contiguous")
        dy = dy.view(-1, D)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the gradient to add to as out")
        with binding.allocating_on(stream):
            out = torch.empty(rows, D, dtype=out_dtype or dy.dtype, device=dy.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out must be {out_dtype}, got {out.dtype}")
    elif out.dim() != 2 or out.shape[0] != rows:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected ({rows}, {D})")
    with binding.allocating_on(stream):
        workspace = torch.empty(max(16, binding.embedding_grad_workspace(flat.numel(), rows, D)),
                                dtype=torch.uint8, device=dy.device)
    binding.embedding_grad(dy, flat, out, workspace, scale, first_row, accumulate, stream)
    return out
