"""A layer's activation, gated or not, whose inputs are kept in 8 bits for the
backward pass.

    forward:  h = act(gate) * up          (act(gate) without up)
    backward: dgate = dh * up^ * act'(gate^),  dup = dh * act(gate^)

where gate^ and up^ are what the kept codes stand for: e4m3 with one fp32 scale
per 128 values of a row, as `fp8.quantize` makes them, a byte a value instead of
two or four.  They are made in the forward pass's one reading of its inputs.
All arithmetic is in fp32, rounded once to the result's type.

    h, kept = activation.forward(gate, up, kind="silu", save=True)
    dgate, dup = activation.backward(dh, kept)
"""
from __future__ import annotations

import torch

from . import binding
from .fp8 import Fp8Tensor

KINDS = {"relu": binding.WC_RELU, "silu": binding.WC_SILU, "gelu": binding.WC_GELU}


class Kept:
    """What a forward pass keeps: the kind of activation, and gate and up (None
    without one) as Fp8Tensors [rows, columns]."""

    __slots__ = ("kind", "gate", "up")

    def __init__(self, kind: str, gate: Fp8Tensor, up: Fp8Tensor | None):
        self.kind, self.gate, self.up = kind, gate, up


def _kind(kind: str) -> int:
    if kind not in KINDS:
        raise ValueError(f"kind must be one of {', '.join(KINDS)}, got {kind!r}")
    return KINDS[kind]


def forward(gate: torch.Tensor, up: torch.Tensor | None = None, kind: str = "silu", save: bool = False,
            out: torch.Tensor | None = None, stream=None):
    """h of gate's shape and type; with save, (h, Kept).  kind: "relu", "silu" or
    "gelu" (its tanh form).  gate, up, out: float32 or bfloat16, matrices whose rows
    are consecutive values, or contiguous tensors [.., columns]; out may be gate
    or up, and shares no other memory with them."""
    h, g, u = binding.on_stream(stream, gate.device, binding.calls().activation, gate, up, _kind(kind), save, out)
    if not save:
        return h
    return h, Kept(kind, Fp8Tensor._made(g), None if u is None else Fp8Tensor._made(u))


def backward(dh: torch.Tensor, kept: Kept, stream=None):
    """(dgate, dup) of dh's shape and type (which need not be the forward pass's);
    dup is None without a gate."""
    return binding.on_stream(stream, dh.device, binding.calls().activation_grad, dh, _kind(kept.kind),
                             kept.gate._parts, None if kept.up is None else kept.up._parts)
