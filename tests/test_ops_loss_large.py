"""Cross entropy of large logits, as a run that diverges has them: a token whose logits one
column decides has that column's logit as its log-sum, and gradients of exactly 1 there and
-1 at its target, however large the logits are."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, ULP, close, strided

pytestmark = pytest.mark.gpu

SCALES = [1e4, 1e6, 1e8, 5e9, 1e20]


def decided(dev, T, V, D, scale, seed):
    """x, w, y with logits of about `scale`, each row's largest so far above the others that
    no rounding of a logit and no other exponential shows beside it; the 64-bit logits, the
    columns of the largest, and the bound of what a logit may be off by."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device=dev) * D ** -0.5).bfloat16()
    top = torch.randint(0, V, (T,), generator=g, device=dev)
    # (a push of some 8 standard deviations towards a row of w; columns of one value lie on a line)
    x = torch.randn(T, D, generator=g, device=dev) + 8 * D ** 0.5 * w[top].float() / w[top].float().norm(dim=1, keepdim=True)
    x = (x * scale).bfloat16()
    s = x.double() @ w.double().t()
    best, top = s.max(1)
    y = (top + torch.randint(1, V, (T,), generator=g, device=dev)) % V
    off = (D + 16) * 2 * ULP * (x.double().abs() @ w.double().abs().t()).amax(1)
    second = s.scatter(1, top[:, None], -float("inf")).amax(1)
    assert bool((best - second > 2 * off + 110).all())     # exp(-110) is below 2^-149
    return x, w, y, s, top, off


def check(x, w, y, s, top, off, g, losses, lse, dx, dw):
    T, V = s.shape
    best = s.amax(1)
    round_s = 4 * ULP * (best.abs() + s.abs().amax(1))
    close(lse, best, off + round_s, "lse")
    want = best - s.gather(1, y[:, None])[:, 0]
    close(losses, want, 2 * off + round_s + want * 4 * ULP, "losses")
    if dx is None:
        return
    d = torch.zeros(T, V, dtype=torch.float64, device=x.device)
    d.scatter_(1, top[:, None], 1.0)
    d.scatter_(1, y[:, None], -1.0)
    d *= torch.as_tensor(g, dtype=torch.float64, device=x.device).reshape(-1, 1)
    # (g in bf16 where it is a token's own; a product of two terms, then the type)
    own = HALF_STEP[torch.bfloat16] * 1.01 if torch.is_tensor(g) else 4 * ULP
    want, terms = d @ w.double(), d.abs() @ w.double().abs()
    close(dx, want, terms * own + want.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-37, "dx")
    want, terms = d.t() @ x.double(), d.abs().t() @ x.double().abs()
    close(dw, want, terms * (own + (T + 16) * 2 * ULP) + want.abs() * HALF_STEP[dw.dtype] * 1.01 + 1e-37, "dw")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T,V,D", [(5, 700, 64), (16, 5000, 1000), (300, 700, 64), (260, 1003, 333), (700, 300, 1024),
                                   (70, 20001, 128),
                                   # rows whose products are summed in several chunks
                                   (5, 700, 2048), (300, 700, 2500), (130, 1003, 4104), (600, 900, 4500), (16, 300, 9001),
                                   (1000, 1500, 2048)])
def test_a_column_that_decides(dev, T, V, D, scale):
    from weight_communication_gb300 import binding, loss
    x, w, y, s, top, off = decided(dev, T, V, D, scale, seed=T)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    for g in (0.25, torch.rand(T, device=dev)):
        dx, dw = loss.cross_entropy_grad(x, w, y, lse, g, dw_dtype=torch.float32)
        check(x, w, y, s, top, off, g, losses, lse, dx, dw)
    # a target that decides has no loss and no gradient
    losses, lse = loss.cross_entropy(x, w, top, save=True)
    assert bool((losses == 0).all())
    dx, dw = loss.cross_entropy_grad(x, w, top, lse, 1.0)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    assert binding.wait_timeouts() == 0


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("V,D", [(700, 64), (5001, 333), (1200, 2048), (300, 4104), (300, 9001)])
def test_losses_of_few_tokens(dev, T, V, D, scale):
    from weight_communication_gb300 import loss
    x, w, y, s, top, off = decided(dev, T, V, D, scale, seed=T + 10)
    for rows in (w, strided(w, D + 3, 1)):
        losses, lse = loss.cross_entropy(x, rows, y, save=True)
        check(x, w, y, s, top, off, None, losses, lse, None, None)
        assert bool((loss.cross_entropy(x, rows, top) == 0).all())


@pytest.mark.parametrize("T", [3, 40])
def test_finite_and_infinite_logits_of_a_row(dev, T):
    """Columns without a logit (-infinity) beside large ones, columns that are all without one."""
    from weight_communication_gb300 import loss
    w = torch.zeros(600, 8, device=dev, dtype=torch.bfloat16)
    w[:, 0] = -float("inf")
    w[300:, 0] = -2.0 ** 33
    w[577, 0] = -2.0 ** 32
    x = torch.zeros(T, 8, device=dev, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    y = torch.full((T,), 400, device=dev)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    assert bool((lse == -2.0 ** 32).all()) and bool((losses == 2.0 ** 32).all())
    _, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0, dw_dtype=torch.float32, needs_dx=False)
    want = torch.zeros(600, 8, device=dev)
    want[577, 0], want[400, 0] = T, -T
    assert torch.equal(dw, want)
    assert bool((loss.cross_entropy(x, w, torch.full((T,), 577, device=dev)) == 0).all())


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("V,D", [(700, 64), (5001, 333), (20001, 130), (1200, 512), (2001, 1000), (1200, 2048), (900, 4096), (333, 4090),
                                 (300, 4104), (300, 4500), (9000, 4999), (300, 9001), (200, 30008)])
def test_few_tokens_that_a_column_decides(dev, T, V, D, scale):
    from weight_communication_gb300 import binding, loss
    x, w, y, s, top, off = decided(dev, T, V, D, scale, seed=T + 20)
    g = 0.25 if T % 2 else torch.rand(T, device=dev)
    first = None
    for rows in (w, strided(w, D + 3, 1), strided(w, (D + 15) // 8 * 8, 8)):
        losses, lse = loss.cross_entropy(x, rows, y, save=True)
        for ld, at in ((D, 0), (D + 5, 3)):
            dw = strided(torch.zeros(V, D, device=dev), ld, at)
            dx, dw = loss.cross_entropy_grad(x, rows, y, lse, g, dw=dw)
            check(x, w, y, s, top, off, g, losses, lse, dx, dw)
            # where rows lie changes no bit of a logit
            first = first or (losses, lse, dx, dw)
            assert all(torch.equal(a, b) for a, b in zip(first, (losses, lse, dx, dw)))
        losses, lse = loss.cross_entropy(x, rows, top, save=True)
        dx, dw = loss.cross_entropy_grad(x, rows, top, lse, 1.0)
        assert bool((losses == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())
    assert binding.wait_timeouts() == 0


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("V,D", [(5000, 256), (700, 2048), (333, 4104)])
def test_padding_beside_a_column_that_decides(dev, T, V, D):
    """A token of padding has a log-sum and no gradient."""
    from weight_communication_gb300 import loss
    x, w, y, s, top, off = decided(dev, T, V, D, 1e6, seed=T + 30)
    y[T // 2] = V + 3
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    best = s.amax(1)
    close(lse, best, off + 4 * ULP * (best.abs() + s.abs().amax(1)), "lse")
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0)
    live = torch.arange(T, device=dev) != T // 2
    assert float(losses[T // 2]) == 0.0 and bool((dx[T // 2] == 0).all())
    if T > 1:
        check(x[live], w, y[live], s[live], top[live], off[live], 1.0, losses[live], lse[live], dx[live], dw)
    else:
        assert bool((dw == 0).all())


@pytest.mark.parametrize("T,V,D", [(1, 1100000, 2049), (3, 1100000, 2049), (2, 1100000, 2048), (2, 600000, 4104), (3, 600000, 4105)])
def test_offsets_beyond_32_bits_for_few_tokens(dev, T, V, D):
    """Weights of 2^31 values and more, of which all rows but a few are 0."""
    from weight_communication_gb300 import loss
    g = torch.Generator(device=dev)
    g.manual_seed(T + D)
    rows = torch.tensor([0, 5, V // 2, (1 << 31) // D, (1 << 31) // D + 1, V - 2, V - 1], device=dev)
    w = torch.zeros(V, D, device=dev, dtype=torch.bfloat16)
    w[rows] = torch.randn(7, D, generator=g, device=dev).bfloat16()
    x = (torch.randn(T, D, generator=g, device=dev) * 0.2).bfloat16()
    at = torch.arange(T, device=dev) + 3
    losses, lse = loss.cross_entropy(x, w, rows[at], save=True)
    dx, dw = loss.cross_entropy_grad(x, w, rows[at], lse, 1.0)
    s = x.double() @ w[rows].double().t()
    want = torch.log(torch.exp(s).sum(1) + (V - 7))
    off = (D + 16) * 2 * ULP * (x.double().abs() @ w[rows].double().abs().t()).amax(1) + (s.abs().amax(1) + 200) * 4 * ULP
    close(lse, want, off, "lse")
    close(losses, want - s.gather(1, at[:, None])[:, 0], 2 * off, "losses")
    d = torch.exp(s - want[:, None])
    off_d = d * (3 * off[:, None] + HALF_STEP[torch.bfloat16]) * 1.01
    d.scatter_add_(1, at[:, None], torch.full((T, 1), -1.0, device=dev, dtype=torch.float64))
    off_d += d.abs() * HALF_STEP[torch.bfloat16] * 1.01
    for got, total, bound, what in ((dx, d @ w[rows].double(), off_d @ w[rows].double().abs(), "dx"),
                                    (dw[rows], d.t() @ x.double(), off_d.t() @ x.double().abs(), "dw")):
        close(got, total, bound + total.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-37, what)
    # all other rows have the same gradient: the tokens by 1 / sum
    other = (x.double() / torch.exp(want)[:, None]).sum(0)
    bound = (x.double().abs() / torch.exp(want)[:, None]).sum(0) * (3 * off.max() + HALF_STEP[torch.bfloat16] * 2.02) + 1e-37
    for r in (1, V // 2 + 1, (1 << 31) // D - 1, (1 << 31) // D + 2, V - 3):
        close(dw[r], other, bound, f"row {r}")
