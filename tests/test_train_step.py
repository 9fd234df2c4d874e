"""The training step that runs lookup, 8-bit layers, qgZ, clipping and update
together."""
import math

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_loss_falls_and_the_gradient_is_clipped(dev):
    from weight_communication_gb300.train_step import TrainStep, batch
    model = TrainStep(vocab=203, width=96, hidden=200, ranks=4, lr=1.0, max_norm=0.5)
    losses, stats = [], []
    for i in range(30):
        loss, st = model.step(*batch(203, 4, 512, i))
        losses.append(float(loss))
        stats.append(st.tolist())
    assert losses[0] > 0.7 * math.log(203)
    assert losses[-1] < 0.8 * losses[0]
    for norm, coef in stats:
        assert norm > 0 and coef == pytest.approx(min(1.0, 0.5 / (norm + 1e-6)), rel=1e-6)
    assert any(coef < 1 for _, coef in stats)


def test_rank_gradient_against_differences(dev):
    """The bucket's gradients are those of the loss, up to what 8 bits round:
    the change of the loss along the gradient's own direction."""
    from weight_communication_gb300.train_step import TrainStep, batch
    model = TrainStep(vocab=130, width=64, hidden=144, ranks=1, seed=3)
    ids, targets = batch(130, 1, 700, 0)
    model.rank_gradient(0, ids[0], targets[0])
    for name in ("table", "up", "down", "head"):
        g = model.grads[0][name].float().clone()
        w = model.weights[name]
        kept = w.clone()
        step = 0.05 * float(w.norm()) / float(g.norm())
        ends = []
        for sign in (1.0, -1.0):
            w.copy_(kept + sign * step * g)
            model.table.copy_(model.weights["table"])
            for n, lin in (("up", model.up), ("down", model.down), ("head", model.head)):
                lin.load(model.weights[n])
            ends.append(float(model.rank_gradient(0, ids[0], targets[0])))
        w.copy_(kept)
        slope = (ends[0] - ends[1]) / (2 * step)
        want = float(g.norm()) ** 2
        # e4m3 keeps 4 significant bits: 2^-4 of each factor, and the loss is
        # curved over a step of a twentieth of the weights
        assert slope == pytest.approx(want, rel=0.15), name


def test_same_bits_every_run(dev):
    from weight_communication_gb300.train_step import TrainStep, batch
    runs = []
    for _ in range(2):
        model = TrainStep(vocab=203, width=96, hidden=200, ranks=2)
        for i in range(3):
            _, stats = model.step(*batch(203, 2, 300, i))
        runs.append((model.reducer.out.clone(), stats.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
