"""Activations kept in 8 bits: forward, what is kept, and backward against 64-bit
formulas; strides, types, empty and non-finite inputs, differences, graphs."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, ULP, act, close, kept, strided

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 5504), (3, 127), (17, 128), (16, 129), (5, 8), (33, 264), (100, 1003), (257, 520), (2, 40000)]


def inputs(dev, rows, cols, dtype, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = lambda s: (torch.randn(rows, cols, generator=g, device=dev) * s).to(dtype)  # noqa: E731
    return n(2.0), n(1.0), n(1e-2)


def check(kind, gate, up, dh, h, saved, dgate, dup):
    t, tb = h.dtype, dgate.dtype
    f, _, off, _ = act(kind, gate)
    u = up.double() if up is not None else torch.ones_like(f)
    # (results below the smallest normal number may be lost)
    close(h, f * u, u.abs() * off + (f * u).abs() * (2 * ULP + HALF_STEP[t] * 1.01) + 1e-37, "h")
    if saved is None:
        return
    g8 = kept(gate)
    f, d, off_f, off_d = act(kind, g8)
    u8 = kept(up) if up is not None else torch.ones_like(f)
    w = dh.double()
    fuzz = 4 * ULP + HALF_STEP[tb] * 1.01
    close(dgate, w * u8 * d, (w * u8).abs() * off_d + (w * u8 * d).abs() * fuzz + 1e-37, "dgate")
    if up is not None:
        close(dup, w * f, w.abs() * off_f + (w * f).abs() * fuzz + 1e-37, "dup")


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(dev, rows, cols, kind):
    from weight_communication_gb300 import activation, fp8
    for dtype in (torch.bfloat16, torch.float32):
        gate, up, dh = inputs(dev, rows, cols, dtype)
        for u in (None, up):
            h, saved = activation.forward(gate, u, kind=kind, save=True)
            dgate, dup = activation.backward(dh, saved)
            assert (dup is None) == (u is None) == (saved.up is None)
            check(kind, gate, u, dh, h, saved, dgate, dup)
            assert torch.equal(h, activation.forward(gate, u, kind=kind))
            for x, q in ((gate, saved.gate), (u, saved.up)):
                if x is None:
                    continue
                want, _ = fp8.quantize(x)
                assert torch.equal(q.codes.view(torch.uint8), want.codes.view(torch.uint8))
                assert torch.equal(q.scales, want.scales)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,ld,offset", [(264, 272, 0), (264, 272, 8), (264, 265, 0), (264, 272, 3), (131, 137, 1),
                                            (1000, 1003, 5)])
def test_rows_that_start_anywhere(dev, dtype, cols, ld, offset):
    from weight_communication_gb300 import activation
    gate, up, dh = inputs(dev, 37, cols, dtype, 1)
    want, saved = activation.forward(gate, up, save=True)
    grads = activation.backward(dh, saved)
    g, u, d = strided(gate, ld, offset), strided(up, ld + 4, offset), strided(dh, ld, offset)
    out = strided(torch.zeros_like(gate), ld, offset)
    h, again = activation.forward(g, u, save=True, out=out)
    assert h is out and torch.equal(h, want)
    assert float(out._base.float().sum()) == pytest.approx(float(h.float().sum()) + 3.0 * (out._base.numel() - h.numel()), rel=1e-4)
    for a, b in zip(activation.backward(d, again), grads):
        assert torch.equal(a, b)


def test_shapes_types_and_places(dev):
    from weight_communication_gb300 import activation
    gate, up, dh = inputs(dev, 24, 136, torch.bfloat16, 2)
    want, saved = activation.forward(gate, up, save=True)
    h, kept3 = activation.forward(gate.view(2, 12, 136), up.view(2, 12, 136), save=True)
    assert h.shape == (2, 12, 136) and torch.equal(h.view(24, 136), want)
    a, b = activation.backward(dh.view(2, 12, 136), kept3)
    assert a.shape == b.shape == (2, 12, 136)
    # fp32 gradients of a bf16 forward pass
    c, d = activation.backward(dh.float(), saved)
    assert c.dtype == d.dtype == torch.float32
    assert torch.equal(c.bfloat16(), a.view(24, 136)) and torch.equal(d.bfloat16(), b.view(24, 136))
    # in place
    g = gate.clone()
    assert activation.forward(g, up, out=g) is g and torch.equal(g, want)
    u = up.clone()
    assert activation.forward(gate, u, out=u) is u and torch.equal(u, want)
    for shape in ((0, 16), (5, 0), (0, 0)):
        e = torch.empty(shape, device=dev)
        h, s = activation.forward(e, e, save=True)
        assert h.shape == shape
        assert all(x.shape == shape for x in activation.backward(e, s))


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_values(dev, kind, dtype):
    from weight_communication_gb300 import activation
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 88.0, -88.0, 100.0, -100.0, 1e4, -1e4, 1e9, -1e9], device=dev)
    gate = v.repeat(128, 10)[:, :130].t().contiguous().to(dtype)   # a value per row: kept to a code's step
    dh = torch.ones_like(gate)
    h, saved = activation.forward(gate, kind=kind, save=True)
    dgate, _ = activation.backward(dh, saved)
    check(kind, gate, None, dh, h, saved, dgate, None)
    big = torch.full((2, 128), 3e38, device=dev).to(dtype)
    big[1] = -big[1]
    h, saved = activation.forward(big, kind=kind, save=True)
    assert torch.equal(h[0], big[0]) and bool((h[1] == 0).all())
    dgate, _ = activation.backward(torch.ones_like(big), saved)
    assert bool((dgate[0] == 1).all()) and bool((dgate[1] == 0).all())


def test_values_that_are_not_finite(dev):
    from weight_communication_gb300 import activation
    gate, up, dh = inputs(dev, 20, 300, torch.bfloat16, 3)
    gate[3, 5] = float("nan")
    gate[4, 200] = float("inf")
    up[5, 290] = float("nan")
    h, saved = activation.forward(gate, up, save=True)
    bad = h.isnan()
    assert bad[3, 5] and bad[5, 290] and int(bad.sum()) == 2 and h[4, 200].isinf()
    dgate, dup = activation.backward(dh, saved)
    for row, cols in ((3, slice(0, 128)), (4, slice(128, 256))):
        assert bool(dgate[row, cols].isnan().all()) and bool(dup[row, cols].isnan().all())
    assert bool(dgate[5, 256:].isnan().all()) and not bool(dup[5].isnan().any())
    assert int(dgate.isnan().sum()) == 128 + 128 + 44 and int(dup.isnan().sum()) == 256


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_against_differences(dev, kind):
    """The gradient is that of the forward pass at what was kept."""
    from weight_communication_gb300 import activation, fp8
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    draw = lambda: torch.randint(-28, 29, (8, 256), generator=g, device=dev).float() / 16  # noqa: E731
    gate, up, dh = draw(), draw(), draw()
    gate[:, ::128] = up[:, ::128] = 1.75
    _, saved = activation.forward(gate, up, kind=kind, save=True)
    dgate, dup = activation.backward(dh, saved)
    gate, up = fp8.dequantize(saved.gate, torch.float32), fp8.dequantize(saved.up, torch.float32)
    step = 2.0 ** -6
    for x, d in ((gate, dgate), (up, dup)):
        ends = []
        for sign in (1, -1):
            x.add_(sign * step)
            ends.append(activation.forward(gate, up, kind=kind).double() * dh.double())
            x.sub_(sign * step)
        slope = (ends[0] - ends[1]) / (2 * step)
        # the third derivative of either is below 2, and fp32 values are near 2:
        # step^2 / 6 * 2 * |up| |dh|, and 2^-23 / step
        assert float((slope - d.double()).abs().max()) < step * step / 3 * 3.1 + 8 * 2.0 ** -23 / step


def test_streams_and_graphs(dev):
    from weight_communication_gb300 import activation
    gate, up, dh = inputs(dev, 65, 1000, torch.bfloat16, 5)
    want, saved = activation.forward(gate, up, save=True)
    grads = activation.backward(dh, saved)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    h, k = activation.forward(gate, up, save=True, stream=s)
    a, b = activation.backward(dh, k, stream=s)
    s.synchronize()
    assert torch.equal(h, want) and torch.equal(a, grads[0]) and torch.equal(b, grads[1])
    graph = torch.cuda.CUDAGraph()
    gate2 = torch.zeros_like(gate)
    with torch.cuda.graph(graph):
        h, k = activation.forward(gate2, up, save=True)
        a, b = activation.backward(dh, k)
    gate2.copy_(gate)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(a, grads[0]) and torch.equal(b, grads[1])
