"""A TensorList stands for its tensors wherever they are, not for the memory
that they had when it was made."""
import copy
import pickle

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", TYPES)
def test_a_tensor_that_moved(dev, dtype):
    """`data` points elsewhere (the earlier memory is kept, so that nothing here
    reads memory that is gone)."""
    from weight_communication_gb300 import gradnorm
    a, b = (torch.full((3000,), 1.0, dtype=dtype, device=dev) for _ in range(2))
    lst = gradnorm.TensorList([a, b])
    earlier = a.detach()
    a.data = torch.full((3000,), 2.0, dtype=dtype, device=dev)
    norm = (3000 * 5.0) ** 0.5
    assert float(gradnorm.norm(lst)) == pytest.approx(norm, rel=1e-6)
    gradnorm.clip(lst, 0.5 * norm)
    assert bool((a == 1.0).all()) and bool((b == 0.5).all()) and bool((earlier == 1.0).all())


def test_a_tensor_of_another_length(dev):
    from weight_communication_gb300 import gradnorm
    flat = torch.full((4000,), 3.0, device=dev)
    a = flat[:16]
    lst, out = gradnorm.TensorList([a]), gradnorm.TensorList([torch.zeros(16, device=dev)])
    a.set_(flat[:100])
    assert float(gradnorm.norm(lst)) == 30.0
    with pytest.raises(RuntimeError, match="values"):
        gradnorm.clip(lst, 1.0, out=out)
    a.set_(flat[::2])
    with pytest.raises(ValueError, match="contiguous"):
        gradnorm.norm(lst)


@pytest.mark.parametrize("how", [copy.deepcopy, lambda t: pickle.loads(pickle.dumps(t))],
                         ids=["deepcopy", "pickle"])
def test_copies_have_their_own_tensors(dev, how):
    from weight_communication_gb300 import gradnorm
    lst = gradnorm.TensorList([torch.full((n,), 2.0, device=dev) for n in (5, 700)])
    c = how(lst)
    assert c.device == lst.device and len(c) == 2
    stats = gradnorm.clip(c, 1.0)
    assert float(stats[1]) < 1 and all(bool((t == 2.0 * stats[1]).all()) for t in c.tensors)
    assert all(bool((t == 2.0).all()) for t in lst.tensors)
