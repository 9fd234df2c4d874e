"""Quantization of rows that start on any element: every remainder of the row
distance by 16 bytes, with NaN in the memory between the rows and after the
last one.  Codes and scales equal the definition's."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from test_ops_fp8 import check_quant, gen
from weight_communication_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(1, 9), (8, 136), (137, 250), (128, 128), (270, 401)])
@pytest.mark.parametrize("pad", range(9))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("square", [False, True])
def test_any_row_distance(dev, M, K, pad, dtype, square):
    ld = K + pad
    flat = torch.full((M * ld + 64,), float("nan"), dtype=dtype, device=dev)
    x = flat[:M * ld].view(M, ld)[:, :K]
    x.copy_(torch.randn(M, K, generator=gen(M + K + pad), device=dev))
    q, qt = (fp8.quantize_weight if square else fp8.quantize)(x, columns=True)
    check_quant(q, x, square)
    check_quant(qt, x.t().contiguous(), square)
