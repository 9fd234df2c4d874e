"""Values back from 8 bits: one product and one rounding, exactly."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (16, 128), (17, 513), (130, 1000), (300, 1003), (257, 24), (3, 5000)])
@pytest.mark.parametrize("square", [False, True])
def test_values(dev, rows, cols, square):
    from weight_communication_gb300 import fp8
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    x = torch.randn(rows, cols, generator=g, device=dev) * 3
    x[rows // 2, cols // 2] = 300.0
    q, qt = (fp8.quantize_weight if square else fp8.quantize)(x, columns=True)
    for m, shape in ((q, (rows, cols)), (qt, (cols, rows))):
        per = m.scales.t().repeat_interleave(m.block_rows, 0)[:m.rows].repeat_interleave(128, 1)[:, :m.cols]
        want = m.codes[:, :m.cols].float() * per
        for dtype in (torch.float32, torch.bfloat16):
            got = fp8.dequantize(m, dtype)
            assert got.shape == shape and got.dtype == dtype and torch.equal(got, want.to(dtype))
            for ld, offset in ((m.cols + 3, 1), (-(-m.cols // 8) * 8 + 8, 0)):
                out = strided(torch.zeros(shape, device=dev, dtype=dtype), ld, offset)
                kept = out._base.clone()
                assert fp8.dequantize(m, out=out) is out and torch.equal(out, want.to(dtype))
                out.copy_(strided(torch.zeros(shape, device=dev, dtype=dtype), ld, offset))
                assert torch.equal(out._base, kept)   # nothing beside it is written


def test_every_code_and_scale(dev):
    from weight_communication_gb300 import fp8
    codes = torch.arange(256, dtype=torch.uint8, device=dev).repeat(3, 1).view(torch.float8_e4m3fn)
    scales = torch.tensor([[1.0, 2.0 ** -126, float("nan")], [3e38, 0.0, 1.1]], device=dev)
    got = fp8.dequantize(fp8.Fp8Tensor(codes, scales, 3, 256), torch.float32)
    want = codes.float() * scales.t().repeat_interleave(128, 1)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0, 8.0, -8.0), want.nan_to_num(7.0, 8.0, -8.0))


def test_empty_stream_and_graph(dev):
    from weight_communication_gb300 import fp8
    assert fp8.dequantize(fp8.Fp8Tensor.empty(0, 5, device=dev)).shape == (0, 5)
    assert fp8.dequantize(fp8.Fp8Tensor.empty(5, 0, device=dev)).shape == (5, 0)
    x = torch.randn(100, 300, device=dev)
    q, _ = fp8.quantize(x)
    want = fp8.dequantize(q)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    got = fp8.dequantize(q, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.dequantize(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
