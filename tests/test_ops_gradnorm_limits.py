"""The coefficient where max_norm / (norm + eps) is no number by itself: an
infinite norm gives 0 whatever the bound, and nothing to clip gives 1."""
import math

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, math.inf])
def test_infinite_norm(dev, dtype, max_norm):
    from weight_communication_gb300 import gradnorm
    x = torch.ones(5000, dtype=dtype, device=dev)
    x[77] = math.inf
    out = torch.full_like(x, 9.0)
    assert gradnorm.clip([x], max_norm, out=[out]).tolist() == [math.inf, 0.0]
    assert math.isnan(float(out[77])) and float(out.nan_to_num(0.0).abs().max()) == 0.0


@pytest.mark.parametrize("max_norm", [0.0, 1.0, math.inf])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_zero_norm(dev, max_norm, eps):
    """min(1, max_norm / eps) where eps is not 0, and 1 where it is."""
    from weight_communication_gb300 import gradnorm
    want = min(1.0, max_norm / eps) if eps else 1.0
    x = torch.zeros(5000, device=dev)
    out = torch.full_like(x, 9.0)
    assert gradnorm.clip([x], max_norm, out=[out], eps=eps).tolist() == [0.0, want]
    assert bool((out == 0).all())
    assert gradnorm.clip([x], max_norm, eps=eps).tolist() == [0.0, want] and bool((x == 0).all())
    assert gradnorm.clip([x[:0]], max_norm, eps=eps).tolist() == [0.0, want]


@pytest.mark.parametrize("max_norm", [0.0, math.inf])
def test_bounds_at_both_ends(dev, max_norm):
    from weight_communication_gb300 import gradnorm
    x = torch.full((5000,), 2.0, device=dev)
    coef = 0.0 if max_norm == 0 else 1.0
    assert gradnorm.clip([x], max_norm, eps=0.0).tolist() == [float(torch.tensor(2.0 * 5000 ** 0.5)), coef]
    assert bool((x == 2.0 * coef).all())
    x[5] = math.nan
    assert math.isnan(float(gradnorm.clip([x], max_norm)[1]))
