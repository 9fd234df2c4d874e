"""Gradients of the cross entropy whose sums run over many tokens or a large vocabulary,
against 64-bit formulas, and against differences along the gradient itself."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, ULP, close
from test_ops_loss import inputs, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [8192, 16385, 140001, 1 << 20])
def test_what_sums_lose_does_not_grow_with_the_tokens(dev, T, dtype, accumulate):
    """Terms of one sign: two rows of weight that are 0 have probabilities of a half each."""
    from weight_communication_gb300 import binding, loss
    g = torch.Generator(device=dev)
    g.manual_seed(T)
    x = torch.rand(T, 72, generator=g, device=dev).add_(0.5).bfloat16()
    w = torch.zeros(2, 72, device=dev, dtype=torch.bfloat16)
    y = torch.zeros(T, device=dev, dtype=torch.int64)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    old = torch.rand(2, 72, generator=g, device=dev).to(dtype)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0, dw=old.clone(), accumulate=accumulate)
    torch.cuda.synchronize()
    assert binding.wait_timeouts() == 0
    half = 0.5 * x.double().sum(0)
    # d is exact; 512 steps of 16 values to a chunk, each of which may lose an ulp of what is
    # summed so far, and a rounding for each chunk that is added; then the result's
    off = half * (512 * 2 ** -23 + -(-T // 8192) * ULP)
    want = torch.stack([-half, half]) + (old.double() if accumulate else 0.0)
    close(dw, want, off + want.abs() * HALF_STEP[dtype] * 1.01, "dw")
    assert bool((dx == 0).all())


@pytest.mark.parametrize("T,V,D", [(20000, 700, 72), (8192, 40000, 264), (40001, 1003, 130), (3500, 60000, 72)])
def test_many_terms(dev, T, V, D):
    from weight_communication_gb300 import binding, loss
    x, w, y = inputs(dev, T, V, D, seed=12)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0 / T, dw_dtype=torch.float32)
    again = loss.cross_entropy_grad(x, w, y, lse, 1.0 / T, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    assert binding.wait_timeouts() == 0
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    want, off = reference(x, w, y, 1.0 / T)
    close(losses, want[0], off[0] + want[0].abs() * 2 * ULP, "losses")
    close(dx, want[2], off[2] + want[2].abs() * HALF_STEP[dx.dtype] * 1.01 + 1e-37, "dx")
    close(dw, want[3], off[3] + want[3].abs() * ULP + 1e-37, "dw")


@pytest.mark.parametrize("T,V,D", [(64, 300, 128), (3, 300, 128), (2, 300, 4104), (300, 1000, 1100)])
def test_gradient_against_differences_along_itself(dev, T, V, D):
    """The loss's change along the gradient's own direction is the gradient's length: a gradient of
    another sign, length or place does not pass (along a random direction nearly all do)."""
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, T, V, D, padding=T > 3, seed=13)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    g = torch.rand(T, device=dev)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, g, dw_dtype=torch.float32)
    value = lambda a, b: float((loss.cross_entropy(a, b, y).double() * g.double()).sum())  # noqa: E731
    for arg, d in ((x, dx), (w, dw)):
        # a fiftieth of the values that the gradient is mostly of: all, or the targets' rows
        rows = arg if arg is x else arg[y[(y >= 0) & (y < V)].unique()]
        step = 0.02 * float(rows.double().norm()) * d.double() / float(d.double().norm())
        plus, minus = (arg.double() + step).bfloat16(), (arg.double() - step).bfloat16()
        slope = value(plus, w) - value(minus, w) if arg is x else value(x, plus) - value(x, minus)
        moved = plus.double() - minus.double()
        # the loss's third derivative over such a step (0.003 of the slope over 60 seeds in 64
        # bits), d's rounding to 2^-9, and the ends' middle, off arg by as much
        bound = 0.03
        assert slope == pytest.approx(float((d.double() * moved).sum()), rel=bound)
        for wrong in (-d, 2 * d, 0.5 * d, d.flip(0), d.roll(1, 1)):
            assert slope != pytest.approx(float((wrong.double() * moved).sum()), rel=bound)


@pytest.mark.parametrize("T", [2, 20])
def test_results_have_memory_of_their_own(dev, T):
    """A weight is not updated in place; a gradient beside it in one tensor is."""
    from weight_communication_gb300 import binding, loss
    x, w, y = inputs(dev, T, 300, 64, padding=False, seed=14)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 0.5)
    both = torch.cat([w, torch.zeros_like(w)], 1)
    before = both.clone()
    for out, weight in ((both[:, :64], both[:, :64]), (both[:, 32:96], both[:, :64]), (both.view(-1)[64:64 + 300 * 64].view(300, 64), both[:, :64])):
        for accumulate in (False, True):
            with pytest.raises(binding.WcError, match="dw overlaps w"):
                loss.cross_entropy_grad(x, weight, y, lse, 0.5, dw=out, accumulate=accumulate)
    with pytest.raises(binding.WcError, match="dw overlaps x"):
        loss.cross_entropy_grad(both[:T, 64:], w, y, lse, 0.5, dw=both[:, 64:])
    torch.cuda.synchronize()
    assert torch.equal(both, before)
    dx2, dw2 = loss.cross_entropy_grad(x, both[:, :64], y, lse, 0.5, dw=both[:, 64:])
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(both[:, :64], w)
