"""Products with few tiles and a long sum, where a cluster of 2 to 8 CTAs shares
each tile's blocks of K.

Tolerance: that of test_ops_fp8 -- (256 + blocks + 4) u of the sum of
magnitudes, u = 2^-24 -- and one addition more per CTA, 8 at most; for bf16
outputs half of 2^-8 of the result besides, for accumulation one addition
(inside the 4).
"""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from test_ops_fp8 import U, gen, values
from weight_communication_gb300 import binding, fp8

pytestmark = pytest.mark.gpu

SIZES = [(1, 5504, 2048),          # one token, 43 tiles of 16 columns
         (1, 128, 128 * 24),       # one tile
         (7, 1000, 128 * 9 + 3),   # blocks that do not divide, a last one of 3
         (16, 4600, 1003), (20, 300, 5001), (33, 129, 11008), (64, 2048, 2048),
         (65, 1003, 4000), (128, 127, 128 * 26), (200, 700, 3001), (333, 1003, 1501),
         (257, 2049, 2500)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_sum(dev, M, N, K, b_square, dtype):
    g = gen(M * 7 + N * 3 + K)
    a = fp8.quantize(torch.randn(M, K, generator=g, device=dev))[0]
    b = (fp8.quantize_weight if b_square else fp8.quantize)(torch.randn(N, K, generator=g, device=dev))[0]
    A, B = values(a), values(b)
    want, mag = A @ B.t(), A.abs() @ B.abs().t()
    # into a wider buffer, whose other columns stay; rows of 16 bytes and odd ones
    for ld in (-(-N // 8) * 8 + 8, N + 3):
        for accumulate in (False, True):
            wide = torch.randn(M, ld, generator=g, device=dev).to(dtype)
            before = wide.clone()
            got = fp8.matmul(a, b, out=wide[:, :N], accumulate=accumulate)
            total, size = want, mag
            if accumulate:
                total, size = want + before[:, :N].double(), mag + before[:, :N].double().abs()
            tol = (256 + -(-K // 128) + 4 + 8) * U * size
            if dtype == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (total.abs() + tol)
            assert bool(((got.double() - total).abs() <= tol).all())
            assert torch.equal(wide[:, N:], before[:, N:])
            again = before[:, :N].clone()
            assert torch.equal(fp8.matmul(a, b, out=again, accumulate=accumulate), got)
    assert binding.wait_timeouts() == 0


def test_shared_sum_of_a_value_that_is_not_a_number(dev):
    """One block's scale is NaN: its row is, whichever CTA has that block."""
    x = torch.randn(4, 128 * 24, device=dev)
    for at in (0, 128 * 11 + 5, 128 * 24 - 1):
        y = x.clone()
        y[2, at] = float("inf")
        out = fp8.matmul(fp8.quantize(y)[0], fp8.quantize(torch.randn(200, 128 * 24, device=dev))[0])
        assert bool(out[2].isnan().all()) and not bool(out[[0, 1, 3]].isnan().any())


def test_shared_sum_in_a_graph_and_beside_other_work(dev):
    """The clusters of one product while another product runs on a second
    stream: each waits for SMs, none for the other."""
    a = fp8.quantize(torch.randn(1, 4096, device=dev))[0]
    b = fp8.quantize_weight(torch.randn(4096, 4096, device=dev))[0]
    big = fp8.quantize(torch.randn(2048, 4096, device=dev))[0]
    want, wide = fp8.matmul(a, b), fp8.matmul(big, b)
    s, t = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    outs = [torch.empty_like(want) for _ in range(20)]
    more = [torch.empty_like(wide) for _ in range(4)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for o in outs:
                fp8.matmul(a, b, out=o)
        graph.replay()
    for o in more:
        fp8.matmul(big, b, out=o, stream=t)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(o, wide) for o in more)
    assert binding.wait_timeouts() == 0
