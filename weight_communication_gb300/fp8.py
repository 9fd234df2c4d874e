"""Linear layers in 8-bit floating point (e4m3) with a scale per block of 128.

A matrix is held as e4m3 codes and fp32 scales: one scale for every 128 values
along the axis that a product sums over (activations and gradients), or one
for every 128 x 128 (weights).  `quantize` and `quantize_weight` make such
matrices, `matmul` multiplies two of them on the tensor cores with fp32 sums,
and `Fp8Linear` composes them into a layer's forward and backward pass:

    lin = Fp8Linear(weight)                    # [N, K] bf16 or fp32
    y = lin.forward(x)                         # x W^T
    y, saved = lin.forward(x, save=True)       # training
    dx, dw = lin.backward(dy, saved)           # dy W, dy^T x (fp32)
    lin.load(weight)                           # after an update of the weights
"""
from __future__ import annotations

import torch

from . import binding

BLOCK = 128


def _ceil(n: int, m: int) -> int:
    return -(-n // m) * m


class Fp8Tensor:
    """A matrix [rows, cols] in 8 bits.

    codes  : float8_e4m3fn [rows, >= cols], rows a multiple of 16 bytes apart
    scales : float32 [ceil(cols / 128), >= rows] (block_rows 1) or
             [ceil(cols / 128), >= ceil(rows / 128)] (block_rows 128)
    Row r, column c stands for codes[r, c] * scales[c // 128, r // block_rows].
    The two tensors are checked here, once; don't resize them afterwards.
    """

    __slots__ = ("_codes", "_scales", "_buffer", "_scales_at", "rows", "cols", "block_rows",
                 "ld_codes", "ld_scales", "device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                 block_rows: int = 1):
        if block_rows not in (1, BLOCK):
            raise ValueError(f"block_rows must be 1 or {BLOCK}, got {block_rows}")
        self.ld_codes, self.ld_scales = binding.fp8_strides(codes, scales, rows, cols, block_rows)
        self._codes, self._scales, self.device = codes, scales, codes.device
        self.rows, self.cols, self.block_rows = rows, cols, block_rows
        self._buffer = None

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, device="cuda") -> "Fp8Tensor":
        """Uninitialised, codes and scales in one allocation.  The scales of a
        block start on 16 bytes, where a product fetches them four at a time."""
        t = cls.__new__(cls)
        t.rows, t.cols, t.block_rows = rows, cols, block_rows
        t.ld_codes, t.ld_scales = _ceil(cols, 16), _ceil(-(-rows // block_rows), 4)
        t._scales_at = _ceil(rows * t.ld_codes, 16)
        t._buffer = torch.empty(t._scales_at + -(-cols // BLOCK) * t.ld_scales * 4,
                                dtype=torch.uint8, device=device)
        t._codes = t._scales = None
        t.device = t._buffer.device
        return t

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = (self._buffer[:self.rows * self.ld_codes].view(torch.float8_e4m3fn)
                           .view(self.rows, self.ld_codes))
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            per = -(-self.rows // self.block_rows)
            self._scales = (self._buffer[self._scales_at:].view(torch.float32)
                            .view(-(-self.cols // BLOCK), self.ld_scales)[:, :per])
        return self._scales

    def parts(self) -> tuple:
        """Addresses and strides, as the C calls take them."""
        if self._buffer is not None:
            at = self._buffer.data_ptr()
            return at, self.ld_codes, at + self._scales_at, self.ld_scales
        return self._codes.data_ptr(), self.ld_codes, self._scales.data_ptr(), self.ld_scales


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
    if x.dim() != 2:
        raise ValueError(f"x must be a matrix, got shape {tuple(x.shape)}")
    if not (rows or columns):
        raise ValueError("neither rows nor columns asked for")
    M, K = x.shape
    with binding.allocating_on(stream):
        q = Fp8Tensor.empty(M, K, block_rows, x.device) if rows else None
        qt = Fp8Tensor.empty(K, M, block_rows, x.device) if columns else None
    _quantize_into(x, q, qt, block_rows, stream)
    return q, qt


_NO_PARTS = (None, 0, None, 0)


def _quantize_into(x, q, qt, block_rows, stream):
    binding.fp8_quant_parts(x, q.parts() if q is not None else _NO_PARTS,
                            qt.parts() if qt is not None else _NO_PARTS, block_rows == BLOCK, stream)


def matmul(a: Fp8Tensor, b: Fp8Tensor, out: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
           stream=None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in bf16 or fp32, a new tensor
    or `out`; with accumulate, added to what `out` holds."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    device = a.device
    if b.device != device:
        raise ValueError(f"b is on {b.device}, expected {device}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the matrix to add to as out")
        with binding.allocating_on(stream):
            out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=device)
    elif out.dim() != 2 or tuple(out.shape) != (a.rows, b.rows):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected ({a.rows}, {b.rows})")
    binding.fp8_matmul_parts(a.parts(), a.block_rows, b.parts(), b.block_rows, a.rows, b.rows,
                             a.cols, device, out, accumulate, stream)
    return out


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
        if tuple(weight.shape) != (self.N, self.K):
            raise ValueError(f"weight has shape {tuple(weight.shape)}, expected ({self.N}, {self.K})")
        _quantize_into(weight, self.w, self.wt, BLOCK, stream)

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
        q, qt = quantize(dy, columns=True, stream=stream)
        dx = matmul(q, self.wt, out_dtype=dx_dtype, stream=stream)
        dw = matmul(qt, saved, out=dw, out_dtype=dw_dtype, accumulate=accumulate, stream=stream)
        return dx, dw
