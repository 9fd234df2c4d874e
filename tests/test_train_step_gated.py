"""The gated training step: lookup, norms, gated 8-bit layers, the loss without
logits, qgZ, clipping and update, in one run."""
import math

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_runs(dev):
    from weight_communication_gb300 import binding
    from weight_communication_gb300.train_step import GatedTrainStep, batch
    model = GatedTrainStep(vocab=203, width=96, hidden=200, ranks=4, lr=0.5, max_norm=0.5)
    before = model.master.clone()
    for i in range(5):
        loss, stats = model.step(*batch(203, 4, 512, i))
        norm, coef = stats.tolist()
        assert math.isfinite(float(loss)) and norm > 0
        assert coef == pytest.approx(min(1.0, 0.5 / (norm + 1e-6)), rel=1e-6)
    assert binding.wait_timeouts() == 0
    for name, w in model.weights.items():
        assert bool(w.isfinite().all()) and not torch.equal(w, model._named(before)[name]), name


def test_rank_gradient_against_differences(dev):
    """The bucket's gradients are those of the loss, up to what 8 bits round:
    the change of the loss along the gradient's own direction."""
    from weight_communication_gb300.train_step import GatedTrainStep, batch
    model = GatedTrainStep(vocab=130, width=64, hidden=144, ranks=1, seed=3)
    ids, targets = batch(130, 1, 700, 0)
    model.rank_gradient(0, ids[0], targets[0])
    # (the calls below write their own gradients, at other weights)
    grads = {name: model.grads[0][name].float().clone() for name in model.shapes}
    for name, g in grads.items():
        w = model.weights[name]
        kept = w.clone()
        step = 0.05 * float(w.norm()) / float(g.norm())
        ends = []
        for sign in (1.0, -1.0):
            w.copy_(kept + sign * step * g)
            model.load()
            ends.append(float(model.rank_gradient(0, ids[0], targets[0])))
        w.copy_(kept)
        slope = (ends[0] - ends[1]) / (2 * step)
        want = float(g.norm()) ** 2
        # e4m3 keeps 4 significant bits: 2^-4 of each factor, and the loss is
        # curved over a step of a twentieth of the weights
        assert slope == pytest.approx(want, rel=0.15), name


def test_same_bits_every_run(dev):
    from weight_communication_gb300.train_step import GatedTrainStep, batch
    runs = []
    for _ in range(2):
        model = GatedTrainStep(vocab=203, width=96, hidden=200, ranks=2)
        for i in range(3):
            _, stats = model.step(*batch(203, 2, 300, i))
        runs.append((model.reducer.out.clone(), stats.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_gradients_against_autograd(dev):
    """Every gradient of the chain of calls against autograd in 64 bits of the same
    model without 8 bits: the directions agree."""
    from weight_communication_gb300.train_step import GatedTrainStep, batch
    model = GatedTrainStep(vocab=300, width=128, hidden=256, ranks=1, seed=5)
    ids, targets = batch(300, 1, 600, 1)
    ids, targets = ids[0], targets[0]
    loss = model.rank_gradient(0, ids, targets)
    p = {n: w.double().clone().requires_grad_() for n, w in model.weights.items()}

    def rms(t, w):
        return t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    x = p["table"][ids] * model.scale
    n = rms(x, p["norm_in"][0])
    h = torch.nn.functional.silu(n @ p["gate"].t()) * (n @ p["up"].t())
    z = rms(x + h @ p["down"].t(), p["norm_out"][0])
    want = torch.nn.functional.cross_entropy(z @ p["head"].t(), targets)
    want.backward()
    assert float(loss) == pytest.approx(float(want.detach()), rel=0.02)
    for name, w in p.items():
        got, ref = model.grads[0][name].double(), w.grad
        cos = float((got * ref).sum() / (got.norm() * ref.norm()))
        # each of some ten roundings to 4 significant bits is off by 2^-5 rms at most, so
        # the direction by sqrt(10) / 32 = 0.1: a cosine of 0.995
        assert cos > 0.99, (name, cos)
        assert float(got.norm()) == pytest.approx(float(ref.norm()), rel=0.1), name
