"""How the products store: large and small tiles, rows of out that start on 16
bytes and anywhere, ends inside a pass of 32 columns, sums written and added.

Tolerance as in test_ops_fp8.
"""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from test_ops_fp8 import U, gen, values
from weight_communication_gb300 import binding, fp8

pytestmark = pytest.mark.gpu

# (more than 152 tiles of 128 x 128 take tiles of 256 x 256)
SIZES = [(2000, 1300, 130), (1999, 1301, 70), (1665, 1792, 300), (2049, 1537, 128), (130, 263, 257),
         (300, 1112, 140), (129, 31, 64), (257, 161, 200)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stores(dev, M, N, K, b_square, dtype):
    g = gen(M + 3 * N + K)
    a = fp8.quantize(torch.randn(M, K, generator=g, device=dev))[0]
    b = (fp8.quantize_weight if b_square else fp8.quantize)(torch.randn(N, K, generator=g, device=dev))[0]
    A, B = values(a), values(b)
    want, mag = A @ B.t(), A.abs() @ B.abs().t()
    for ld in (-(-N // 8) * 8, -(-N // 8) * 8 + 16, N + 1 + N % 2, N + 2 + N % 2):
        for accumulate in (False, True):
            wide = torch.randn(M, ld, generator=g, device=dev).to(dtype)
            before = wide.clone()
            got = fp8.matmul(a, b, out=wide[:, :N], accumulate=accumulate)
            total, size = want, mag
            if accumulate:
                total, size = want + before[:, :N].double(), mag + before[:, :N].double().abs()
            tol = (256 + -(-K // 128) + 4) * U * size
            if dtype == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (total.abs() + tol)
            assert bool(((got.double() - total).abs() <= tol).all()), (ld, accumulate)
            assert torch.equal(wide[:, N:], before[:, N:]), (ld, accumulate)
    assert binding.wait_timeouts() == 0


@pytest.mark.parametrize("M,N,K", [(1999, 1301, 300), (300, 1112, 140)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_start_anywhere_hold_the_same_bits(dev, M, N, K, dtype):
    g = gen(M)
    a = fp8.quantize(torch.randn(M, K, generator=g, device=dev))[0]
    b = fp8.quantize_weight(torch.randn(N, K, generator=g, device=dev))[0]
    aligned = torch.empty(M, -(-N // 8) * 8, dtype=dtype, device=dev)[:, :N]
    odd = torch.empty(M, N + 1 + N % 2, dtype=dtype, device=dev)[:, :N]
    assert torch.equal(fp8.matmul(a, b, out=aligned), fp8.matmul(a, b, out=odd))
