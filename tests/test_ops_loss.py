"""Cross entropy over a vocabulary without its logits, against 64-bit formulas."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, ULP, close, strided

pytestmark = pytest.mark.gpu


def inputs(dev, T, V, D, wide=True, padding=True, seed=0, sigma=None):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device=dev) * (sigma or D ** -0.5)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device=dev)
    x = torch.randn(T, D, generator=g, device=dev)
    x += torch.rand(T, 1, generator=g, device=dev) * 6 * w[y].float() / max(1e-6, float(w.float().square().sum(1).mean()))
    if padding:
        y[::5] = -100
        y[3::7] = V
    return x.bfloat16(), w, y if wide else y.int()


def reference(x, w, y, dlosses):
    """(values, what each may be off by) of losses, lse, dx, dw."""
    T, D = x.shape
    V = w.shape[0]
    xd, wd = x.double(), w.double()
    s = xd @ wd.t()
    lse = torch.logsumexp(s, 1)
    live = (y >= 0) & (y < V)
    at = torch.where(live, y.long(), 0)
    sy = s.gather(1, at[:, None])[:, 0]
    losses = torch.where(live, lse - sy, 0.0)
    # a logit: every step of the sum may lose an ulp of what it has summed
    off_s = (D + 16) * 2 * ULP * (xd.abs() @ wd.abs().t()).amax(1)
    off_lse = off_s + (lse.abs() + s.abs().amax(1) + 128) * 4 * ULP
    g = torch.where(live, torch.as_tensor(dlosses, device=x.device, dtype=torch.float64).expand(T), 0.0)
    p = torch.exp(s - lse[:, None])
    d = p.clone()
    d.scatter_add_(1, at[:, None], torch.full_like(d[:, :1], -1.0))
    d *= g[:, None]
    # an exponential carries the errors of both logits; then one rounding to bf16
    off_d = g.abs()[:, None] * (p * (off_s + off_lse + (s.abs().amax(1) + lse.abs() + 16) * 4 * ULP)[:, None] + 2 * ULP * p)
    off_d = (off_d + HALF_STEP[torch.bfloat16] * d.abs()) * 1.01
    x0 = torch.where(live[:, None], xd, 0.0)
    dx, dw = d @ wd, d.t() @ x0
    off_dx = off_d @ wd.abs() + (V + 16) * 2 * ULP * (d.abs() @ wd.abs())
    off_dw = off_d.t() @ x0.abs() + (T + 16) * 2 * ULP * (d.abs().t() @ x0.abs())
    return (losses, lse, dx, dw), (off_s + off_lse, off_lse, off_dx, off_dw)


def check(x, w, y, dlosses, losses, lse, dx, dw, old=0.0):
    want, off = reference(x, w, y, dlosses)
    V = w.shape[0]
    assert bool((losses[(y < 0) | (y >= V)] == 0).all())
    close(losses, want[0], off[0] + want[0].abs() * 2 * ULP, "losses")
    close(lse, want[1], off[1], "lse")
    if dx is not None:
        assert bool((dx[(y < 0) | (y >= V)] == 0).all())
        close(dx, want[2], off[2] + want[2].abs() * HALF_STEP[dx.dtype] * 1.01 + 1e-37, "dx")
    if dw is not None:
        total = want[3] + old
        close(dw, total, off[3] + total.abs() * HALF_STEP[dw.dtype] * 1.01 + 1e-37, "dw")


SIZES = [(1, 1, 1), (1, 300, 64), (5, 1000, 72), (2, 256, 8), (128, 128, 64), (256, 256, 256), (257, 511, 130),
         (300, 4000, 520), (1, 32000, 512), (64, 5000, 1001), (777, 1003, 333), (1500, 700, 64), (33, 20011, 96),
         (700, 3, 200)]


@pytest.mark.parametrize("T,V,D", SIZES)
def test_sizes(dev, T, V, D):
    from weight_communication_gb300 import binding, loss
    for wide in (True, False):
        x, w, y = inputs(dev, T, V, D, wide)
        losses, lse = loss.cross_entropy(x, w, y, save=True)
        torch.cuda.synchronize()
        assert binding.wait_timeouts() == 0
        check(x, w, y, 0.0, losses, lse, None, None)
        assert torch.equal(loss.cross_entropy(x, w, y), losses)
        g = torch.randn(T, device=dev) if wide else 1.0 / T
        dx, dw = loss.cross_entropy_grad(x, w, y, lse, g)
        torch.cuda.synchronize()
        assert binding.wait_timeouts() == 0
        assert dx.dtype == dw.dtype == torch.bfloat16
        check(x, w, y, g, losses, lse, dx, dw)
        again = loss.cross_entropy_grad(x, w, y, lse, g)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
