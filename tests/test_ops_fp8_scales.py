"""Products whose scales are far from 1, in every shape of the kernel.

The bound of the other products, (256 + blocks + 4) u of the sum of magnitudes,
holds while the product of the two scales is a normal number; results below
2^-126 add half of 2^-149 for each of a block's two roundings.  A subnormal
product of scales is off by up to 2^-150, and a block's sum is at most
128 * 448^2 < 2^25: 2^-125 per block.  A product that overflows leaves no output
finite.
"""
import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# one shape of the kernel each, and two whose blocks of K a cluster shares
SHAPES = [(1, 300, 2048), (5, 70, 260), (30, 130, 300), (50, 130, 300), (100, 90, 260), (128, 256, 4096),
          (3000, 2900, 260)]


def operand(rows, K, block_rows, scale, largest, seed, dev):
    """Random codes up to `largest`, and scales within a factor of two of `scale`."""
    from weight_communication_gb300 import fp8
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ld = -(-K // 16) * 16
    codes = (torch.rand(rows, ld, generator=g, device=dev) * 2 - 1) * largest
    blocks, per = -(-K // 128), -(-rows // block_rows)
    s = (1.0 + torch.rand(blocks, -(-per // 4) * 4, generator=g, device=dev, dtype=torch.float64)) * scale
    return fp8.Fp8Tensor(codes.to(torch.float8_e4m3fn), s.float(), rows, K, block_rows)


def values(t):
    s = t.scales.double().repeat_interleave(128, 0)[:t.cols].t()
    s = s.repeat_interleave(t.block_rows, 0)[:t.rows]
    return t.codes[:, :t.cols].double() * s


def product(dev, M, N, K, rows_per_scale, scales, largest, extra):
    from weight_communication_gb300 import binding, fp8
    a = operand(M, K, rows_per_scale[0], scales[0], largest, 1, dev)
    b = operand(N, K, rows_per_scale[1], scales[1], largest, 2, dev)
    got = fp8.matmul(a, b, out_dtype=torch.float32)
    A, B = values(a), values(b)
    want, mag = A @ B.t(), A.abs() @ B.abs().t()
    blocks = -(-K // 128)
    tol = (256 + blocks + 4) * U * mag + blocks * (extra + 2.0 ** -149)
    assert bool(torch.isfinite(got).all())
    assert bool(((got.double() - want).abs() <= tol).all())
    assert binding.wait_timeouts() == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("rows_per_scale", [(1, 128), (1, 1)])
# (scale of a, of b, largest code): one huge and one tiny; both tiny and both huge,
# their product just inside the normal numbers (codes so that the sums fit)
@pytest.mark.parametrize("case", [(2.0 ** 110, 2.0 ** -120, 448.0), (2.0 ** -120, 2.0 ** 110, 448.0),
                                  (2.0 ** -63, 2.0 ** -63, 448.0), (2.0 ** -20, 2.0 ** -106, 448.0),
                                  (2.0 ** 62, 2.0 ** 63, 2.0 ** -6), (2.0 ** 110, 2.0 ** 15, 2.0 ** -6)])
def test_scales_with_a_normal_product(dev, M, N, K, rows_per_scale, case):
    product(dev, M, N, K, rows_per_scale, case[:2], case[2], 0.0)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("rows_per_scale", [(1, 128), (1, 1)])
@pytest.mark.parametrize("scales", [(2.0 ** -70, 2.0 ** -70), (2.0 ** -100, 2.0 ** -47), (2.0 ** -120, 2.0 ** -120)])
def test_scales_with_a_subnormal_product(dev, M, N, K, rows_per_scale, scales):
    product(dev, M, N, K, rows_per_scale, scales, 448.0, 2.0 ** -125)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("rows_per_scale", [(1, 128), (1, 1)])
def test_scales_whose_product_overflows(dev, M, N, K, rows_per_scale):
    """Infinite, or not a number (a block's sum of 0, or infinities of both signs)."""
    from weight_communication_gb300 import fp8
    a = operand(M, K, rows_per_scale[0], 2.0 ** 65, 448.0, 1, dev)
    b = operand(N, K, rows_per_scale[1], 2.0 ** 64, 448.0, 2, dev)
    assert not bool(torch.isfinite(fp8.matmul(a, b, out_dtype=torch.float32)).any())
