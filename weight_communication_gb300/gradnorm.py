"""Global gradient norm over many tensors, and clipping.

    norm = sqrt(sum of every x^2),  coef = min(1, max_norm / (norm + eps))

The step between the reduced gradient shards (`qgz`) and the update.  All on
the device: nothing here waits for the GPU, and the norm and the coefficient
come back as a tensor that the update, or a log line some steps later, reads.

    grads = TensorList(model_gradients)         # once: the buffers stay
    stats = clip(grads, max_norm=1.0)           # every step; stats = [norm, coef]
"""
from __future__ import annotations

import torch

from . import binding


class TensorList:
    """A list of gradient tensors (float32 or bfloat16, contiguous, on one GPU,
    of any sizes and at any offsets into larger buffers), checked when it is
    made and at every call, which takes their addresses and lengths as they are
    then.  It keeps the tensors alive."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        self.device = binding.calls().grad_list(self.tensors)

    def __len__(self) -> int:
        return len(self.tensors)


def _listed(tensors) -> TensorList:
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def _run(lst: TensorList, dst: TensorList | None, clipping: bool, max_norm: float, eps: float,
         stats: torch.Tensor | None, stream) -> torch.Tensor:
    if lst.device is None:
        raise ValueError("an empty list has no GPU to run on")
    return binding.on_stream(stream, lst.device, binding.calls().grad_norm, lst.tensors,
                             None if dst is None else dst.tensors, clipping, max_norm, eps, stats)


def norm(tensors, stats: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The norm of a TensorList or a list of tensors, as stats [1] fp32 on the
    device.  Runs on `stream` or the current one."""
    return _run(_listed(tensors), None, False, 0.0, 0.0, stats, stream)


def clip(tensors, max_norm: float, out=None, eps: float = 1e-6,
         stats: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scales the tensors by coef = min(1, max_norm / (norm + eps)), in place
    or into `out` (a TensorList or list of as many tensors of the same lengths;
    their type may be the other one, for instance fp32 gradients for the update
    from bf16 ones).  Returns stats [2] fp32 on the device: norm and coef."""
    lst = _listed(tensors)
    dst = None if out is None else _listed(out)
    if dst is not None:
        if len(dst) != len(lst):
            raise ValueError(f"out has {len(dst)} tensors, expected {len(lst)}")
        if dst.device != lst.device:
            raise ValueError(f"out is on {dst.device}, expected {lst.device}")
    return _run(lst, dst, True, max_norm, eps, stats, stream)
