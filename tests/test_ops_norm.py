"""Root-mean-square norm kept in 8 bits against 64-bit formulas."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, ULP, close, kept, strided

pytestmark = pytest.mark.gpu

EPS = 1e-6
SIZES = [(1, 1), (1, 2048), (3, 127), (9, 128), (700, 64), (5, 257), (33, 512), (1000, 520), (300, 1024), (17, 1503),
         (200, 2048), (65, 4096), (11, 4097), (1300, 8192), (7, 8200), (5, 16384), (3, 16383), (5000, 40)]


def inputs(dev, rows, cols, dtype, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = lambda s, *shape: (torch.randn(*shape, generator=g, device=dev) * s).to(dtype)  # noqa: E731
    x, add, dy, dt = n(2.0, rows, cols), n(0.5, rows, cols), n(1e-2, rows, cols), n(1e-2, rows, cols)
    return x, add, dy, dt, (1 + n(0.2, cols).float()).to(dtype)


def check(x, add, weight, y, total, saved, dy, dtotal, dx, dweight, old=0.0):
    rows, cols = x.shape
    if add is not None:
        assert torch.equal(total, (x.float() + add.float()).to(x.dtype))
    t, w = total.double(), weight.double()
    r = 1 / (t.square().mean(1, keepdim=True) + EPS).sqrt()
    # squares: 16 in turn in a thread, five and up to 32 across; half of that for
    # the root, then a division, a root and two products
    rel = 40 * ULP
    close(y, t * r * w, (t * r * w).abs() * (rel + HALF_STEP[y.dtype] * 1.01) + 1e-37, "y")
    close(saved.rstd, r[:, 0], r[:, 0] * rel, "rstd")
    n, d = kept(total) * r, dy.double()
    wd = d * w
    mean = (wd * n).mean(1, keepdim=True)
    want = r * (wd - n * mean) + (dtotal.double() if dtotal is not None else 0.0)
    # the sum's terms carry n's error and two products, and its order as above
    off = r * (wd.abs() * (rel + 4 * ULP) + n.abs() * ((wd * n).abs().mean(1, keepdim=True) * 100 * ULP + mean.abs() * (2 * rel + 4 * ULP)))
    close(dx, want, off * 1.01 + want.abs() * (2 * ULP + HALF_STEP[dx.dtype] * 1.01) + 1e-37, "dx")
    terms = rows / 152 + 152 + 20   # in turn in a group, its groups by 32, then 32
    close(dweight, (d * n).sum(0) + old, (d * n).abs().sum(0) * (terms * ULP + rel) + HALF_STEP[dweight.dtype] * 1.01 *
          ((d * n).sum(0) + old).abs() + 1e-37, "dweight")


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes(dev, rows, cols, dtype):
    from weight_communication_gb300 import fp8, norm
    x, add, dy, dt, w = inputs(dev, rows, cols, dtype)
    for a, d in ((None, None), (add, dt), (add, None), (None, dt)):
        y, total, saved = norm.rms(x, w, eps=EPS, add=a, save=True)
        assert (total is x) == (a is None)
        dx, dw = norm.rms_grad(dy, w, saved, add=d)
        assert dw.dtype == torch.float32
        check(x, a, w, y, total, saved, dy, d, dx, dw)
        want, _ = fp8.quantize(total)
        assert torch.equal(saved.input.codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(saved.input.scales, want.scales)
        y2, _ = norm.rms(x, w, eps=EPS, add=a)
        assert torch.equal(y, y2)
        dx2, dw2 = norm.rms_grad(dy, w, saved, add=d)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_weight_types_and_accumulation(dev):
    from weight_communication_gb300 import norm
    x, _, dy, _, w = inputs(dev, 300, 1000, torch.bfloat16, 1)
    for weight in (w, w.float()):
        y, total, saved = norm.rms(x, weight, eps=EPS, save=True)
        for dtype in (torch.bfloat16, torch.float32):
            old = torch.randn(1000, device=dev).to(dtype)
            buf = old.clone()
            dx, dw = norm.rms_grad(dy, weight, saved, dweight=buf, accumulate=True)
            assert dw is buf
            check(x, None, weight, y, total, saved, dy, None, dx, dw, old.double())
            dx, dw = norm.rms_grad(dy, weight, saved, dweight=buf)
            check(x, None, weight, y, total, saved, dy, None, dx, dw)
        dx, dw = norm.rms_grad(dy.float(), weight, saved)
        assert dx.dtype == torch.float32
        check(x, None, weight, y, total, saved, dy.float(), None, dx, dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,ld,offset", [(264, 272, 0), (264, 265, 0), (264, 272, 3), (1031, 1037, 1)])
def test_rows_that_start_anywhere(dev, dtype, cols, ld, offset):
    from weight_communication_gb300 import norm
    x, add, dy, dt, w = inputs(dev, 37, cols, dtype, 2)
    y, total, saved = norm.rms(strided(x, ld, offset), strided(w[None], ld, offset)[0], eps=EPS,
                               add=strided(add, ld + 8, offset), save=True)
    dx, dw = norm.rms_grad(strided(dy, ld, offset), w, saved, add=strided(dt, ld, offset + 1))
    check(x, add, w, y, total, saved, dy, dt, dx, dw)


def test_shapes_and_empty(dev):
    from weight_communication_gb300 import norm
    x, add, dy, dt, w = inputs(dev, 24, 136, torch.bfloat16, 3)
    y, t, _ = norm.rms(x, w, add=add, save=True)
    y3, t3, k3 = norm.rms(x.view(4, 6, 136), w, add=add.view(4, 6, 136), save=True)
    assert y3.shape == t3.shape == (4, 6, 136) and torch.equal(y3.view(24, 136), y) and torch.equal(t3.view(24, 136), t)
    dx, _ = norm.rms_grad(dy.view(4, 6, 136), w, k3)
    assert dx.shape == (4, 6, 136)
    e = torch.empty(0, 136, device=dev, dtype=torch.bfloat16)
    y, _, k = norm.rms(e, w, save=True)
    dx, dw = norm.rms_grad(e, w, k)
    assert y.shape == dx.shape == (0, 136) and bool((dw == 0).all())
    old = torch.ones(136, device=dev)
    norm.rms_grad(e, w, k, dweight=old, accumulate=True)
    assert bool((old == 1).all())


def test_extreme_rows(dev):
    """Rows of zeros, of tiny and of not finite values touch no other row."""
    from weight_communication_gb300 import norm
    x, _, dy, _, w = inputs(dev, 8, 300, torch.float32, 4)
    x[1] = 0.0
    x[2] = 1e-25
    x[3, 7] = float("nan")
    x[4, 299] = float("inf")
    y, total, saved = norm.rms(x, w, eps=EPS, save=True)
    dx, dw = norm.rms_grad(dy, w, saved)
    rows = [0, 1, 2, 5, 6, 7]
    assert bool(y[3].isnan().all()) and bool(dx[3].isnan().all())
    assert bool(y[4, 299].isnan()) and bool((y[4, :299] == 0).all())
    t = total[rows].double()
    r = 1 / (t.square().mean(1, keepdim=True) + EPS).sqrt()
    close(y[rows], t * r * w.double(), (t * r * w).abs() * 42 * ULP + 1e-37)
    assert bool(y[rows].isfinite().all()) and bool(dx[rows].isfinite().all())
    # without eps a row of zeros has no norm
    y, _ = norm.rms(x[:2], w, eps=0.0)
    assert bool(y[0].isfinite().all()) and bool(y[1].isnan().all())


def test_gradient_against_differences(dev):
    """At values that 8 bits hold exactly, the gradients are those of the forward pass."""
    from weight_communication_gb300 import norm
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    # 4 significant bits, and a scale of 1.75 / 448 = 2^-8
    x = torch.randint(-7, 8, (6, 256), generator=g, device=dev).float() / 4
    x[:, ::128] = 1.75
    w = 1 + 0.2 * torch.randn(256, generator=g, device=dev)
    dy = torch.randn(6, 256, generator=g, device=dev)
    _, _, saved = norm.rms(x, w, eps=EPS, save=True)
    dx, dw = norm.rms_grad(dy, w, saved)
    value = lambda a, b: float((norm.rms(a, b, eps=EPS)[0].double() * dy.double()).sum())  # noqa: E731
    for arg, d in ((x, dx), (w, dw)):
        u = torch.randn(arg.shape, generator=g, device=dev)
        step = 2.0 ** -8
        plus, minus = arg + step * u, arg - step * u
        slope = (value(plus, w) - value(minus, w) if arg is x else value(x, plus) - value(x, minus))
        want = float((d.double() * (plus.double() - minus.double())).sum())
        # fp32 outputs: 40 ulp of 1536 terms of size 1 in a random sum; curvature step^2
        scale = float(d.double().norm() * (plus - minus).double().norm())
        assert slope == pytest.approx(want, abs=1e-3 * scale)


def test_streams_and_graphs(dev):
    from weight_communication_gb300 import norm
    x, add, dy, dt, w = inputs(dev, 513, 1000, torch.bfloat16, 6)
    y, t, saved = norm.rms(x, w, add=add, save=True)
    dx, dw = norm.rms_grad(dy, w, saved, add=dt)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    y2, t2, k = norm.rms(x, w, add=add, save=True, stream=s)
    dx2, dw2 = norm.rms_grad(dy, w, k, add=dt, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in ((y, y2), (t, t2), (dx, dx2), (dw, dw2)))
    graph = torch.cuda.CUDAGraph()
    x2 = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y2, t2, k = norm.rms(x2, w, add=add, save=True)
        dx2, dw2 = norm.rms_grad(dy, w, k, add=dt)
    x2.copy_(x)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in ((y, y2), (t, t2), (dx, dx2), (dw, dw2)))
