"""Linear layers in 8-bit floating point (e4m3) with a scale per block of 128.

A matrix is held as e4m3 codes and fp32 scales: one scale for every 128 values
along the axis that a product sums over (activations and gradients), or one
for every 128 x 128 (weights).  `quantize` and `quantize_weight` make such
matrices, `dequantize` gives their values back, `matmul` multiplies two of them on the tensor cores with fp32 sums,
and `Fp8Linear` composes them into a layer's forward and backward pass:

    lin = Fp8Linear(weight)                    # [N, K] bf16 or fp32
    y = lin.forward(x)                         # x W^T
    y, saved = lin.forward(x, save=True)       # training
    dx, dw = lin.backward(dy, saved)           # dy W, dy^T x (fp32)
    lin.load(weight)                           # after an update of the weights

Activations and gradients are matrices [tokens, values], their first value on 16
bytes: a batch [.., tokens, values] goes in as x.view(-1, values).

A product scales each block's sum by the product of the two blocks' scales, in
fp32.  That should be a normal number: the largest magnitudes of any two blocks
that meet, multiplied, between 2.4e-33 and 6.8e43.  Below, up to 2^-125 per block
is lost; above, the output is infinite or not a number.
"""
from __future__ import annotations

import torch

from . import binding

BLOCK = 128


class Fp8Tensor:
    """A matrix [rows, cols] in 8 bits.

    codes  : float8_e4m3fn [rows, >= cols], rows a multiple of 16 bytes apart
    scales : float32 [ceil(cols / 128), >= rows] (block_rows 1) or
             [ceil(cols / 128), >= ceil(rows / 128)] (block_rows 128)
    Row r, column c stands for codes[r, c] * scales[c // 128, r // block_rows].
    A copy (copy.deepcopy, pickle, torch.save) has its own codes and scales.
    """

    __slots__ = ("rows", "cols", "block_rows", "device", "_parts")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                 block_rows: int = 1):
        self._set(binding.calls().fp8_view(codes, scales, rows, cols, block_rows))

    @classmethod
    def _made(cls, parts: tuple) -> "Fp8Tensor":
        t = cls.__new__(cls)
        t._set(parts)
        return t

    # The parts (codes and scales, or one buffer of both and None, then the
    # sizes) are the whole state: the calls take the tensors' addresses from
    # them each time.
    def _set(self, parts: tuple) -> None:
        first, _, self.rows, self.cols, self.block_rows = self._parts = parts
        self.device = first.device

    # (codes as bytes: pickle itself does not know tensors of 8-bit floats)
    def __getstate__(self) -> tuple:
        first, scales, *sizes = self._parts
        return (first if scales is None else first.view(torch.uint8), scales, *sizes)

    def __setstate__(self, state: tuple) -> None:
        first, scales, *sizes = state
        self._set((first if scales is None else first.view(torch.float8_e4m3fn), scales, *sizes))

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device="cuda") -> "Fp8Tensor":
        """Uninitialised."""
        return cls._made(binding.calls().fp8_empty(rows, cols, block_rows, torch.device(device)))

    @property
    def codes(self) -> torch.Tensor:
        first, scales = self._parts[:2]
        if scales is not None:
            return first
        ld = -(-self.cols // 16) * 16
        return first[:self.rows * ld].view(torch.float8_e4m3fn).view(self.rows, ld)

    @property
    def scales(self) -> torch.Tensor:
        first, scales = self._parts[:2]
        if scales is not None:
            return scales
        blocks, per = -(-self.cols // BLOCK), -(-self.rows // self.block_rows)
        ld = -(-per // 4) * 4
        return (first[first.numel() - blocks * ld * 4:].view(torch.float32)
                .view(blocks, ld)[:, :per])


def quantize(x: torch.Tensor, rows: bool = True, columns: bool = False, stream=None):
    """x [M, K] (bf16 or fp32) as (x, x^T): an Fp8Tensor [M, K] with a scale per
    128 columns of a row (None unless `rows`) and an Fp8Tensor [K, M] with a
    scale per 128 rows of a column (None unless `columns`), both from one
    reading of x."""
    return _quantize(x, rows, columns, 1, stream)


def quantize_weight(w: torch.Tensor, rows: bool = True, columns: bool = False, stream=None):
    """The same with one scale per 128 x 128, shared by the two layouts."""
    return _quantize(w, rows, columns, BLOCK, stream)


def _quantize(x, rows, columns, block_rows, stream):
    q, qt = binding.on_stream(stream, x.device, binding.calls().fp8_quantize, x, rows, columns,
                              block_rows)
    return (None if q is None else Fp8Tensor._made(q), None if qt is None else Fp8Tensor._made(qt))


def matmul(a: Fp8Tensor, b: Fp8Tensor, out: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
           stream=None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in bf16 or fp32, a new tensor
    or `out`; with accumulate, added to what `out` holds."""
    return binding.on_stream(stream, a.device, binding.calls().fp8_matmul, a._parts, b._parts, out,
                             out_dtype, accumulate)


def dequantize(q: Fp8Tensor, out_dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """What `q` stands for, [rows, cols] in bf16 or fp32: a new tensor or `out`
    (whose rows may start on any value)."""
    return binding.on_stream(stream, q.device, binding.calls().fp8_dequantize, q._parts, out, out_dtype)


class Fp8Linear:
    """y = x W^T with W [N, K] kept in 8 bits (one scale per 128 x 128), in
    both layouts if `training`."""

    def __init__(self, weight: torch.Tensor, training: bool = True, stream=None):
        if weight.dim() != 2:
            raise ValueError(f"weight must be a matrix, got shape {tuple(weight.shape)}")
        self.N, self.K = weight.shape
        self.w, self.wt = quantize_weight(weight, columns=training, stream=stream)

    def load(self, weight: torch.Tensor, stream=None) -> None:
        """Quantizes new values of the weight into the same buffers."""
        binding.on_stream(stream, weight.device, binding.calls().fp8_quantize_into, weight,
                          self.w._parts, None if self.wt is None else self.wt._parts)

    def forward(self, x: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                save: bool = False, stream=None):
        """y [M, N]; with save, also what backward needs of x (x^T in 8 bits)."""
        q, qt = quantize(x, columns=save, stream=stream)
        y = matmul(q, self.w, out_dtype=out_dtype, stream=stream)
        return (y, qt) if save else y

    def backward(self, dy: torch.Tensor, saved: Fp8Tensor, dx_dtype: torch.dtype = torch.bfloat16,
                 dw: torch.Tensor | None = None, dw_dtype: torch.dtype = torch.float32,
                 accumulate: bool = False, stream=None):
        """(dx [M, K], dw [N, K]).  dw: a buffer to write, or with accumulate
        to add to (the gradient of earlier micro-batches)."""
        if self.wt is None:
            raise ValueError("backward needs Fp8Linear(training=True)")
        if dy.dim() != 2 or tuple(dy.shape) != (saved.cols, self.N):
            raise ValueError(f"dy has shape {tuple(dy.shape)}, expected ({saved.cols}, {self.N})")
        if saved.rows != self.K:
            raise ValueError(f"saved is of {saved.rows} columns, the layer has {self.K}: another layer's?")
        q, qt = quantize(dy, columns=True, stream=stream)
        dx = matmul(q, self.wt, out_dtype=dx_dtype, stream=stream)
        dw = matmul(qt, saved, out=dw, out_dtype=dw_dtype, accumulate=accumulate, stream=stream)
        return dx, dw
