"""The training-step calls stand outside autograd: what they write counts as
changed for a backward pass that saved it, and a gradient that ends at one of
them is told of."""
import warnings

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def writes(dev):
    """(name, a call that writes to the tensor it is given): fp32 [12, 16]."""
    from weight_communication_gb300 import embedding, fp8, gradnorm
    ids = torch.arange(12, device=dev)
    table = torch.ones(12, 16, device=dev)
    a, _ = fp8.quantize(table)
    b, _ = fp8.quantize(torch.ones(16, 16, device=dev))
    return {
        "lookup": lambda t: embedding.lookup(table, ids, out=t),
        "grad": lambda t: embedding.grad(table, ids, 12, out=t),
        "grad_accumulate": lambda t: embedding.grad(table, ids, 12, out=t, accumulate=True),
        "matmul": lambda t: fp8.matmul(a, b, out=t),
        "clip": lambda t: gradnorm.clip([t], 1e-3),
        "clip_out": lambda t: gradnorm.clip([table], 1e-3, out=[t]),
        "norm_stats": lambda t: gradnorm.norm([table], stats=t.view(-1)[:1]),
        "clip_stats": lambda t: gradnorm.clip([table.clone()], 1e-3, stats=t.view(-1)[:2]),
    }


NAMES = ["lookup", "grad", "grad_accumulate", "matmul", "clip", "clip_out", "norm_stats", "clip_stats"]


@pytest.mark.parametrize("name", NAMES)
def test_written_tensors_have_a_new_version(dev, name):
    x = torch.ones(12, 16, device=dev, requires_grad=True)
    y = 2 * x
    loss = (y * y).sum()    # saves y
    before = y._version
    writes(dev)[name](y.detach())
    assert y._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_inference_mode(dev, name):
    """They have no version, and are written all the same."""
    with torch.inference_mode():
        t = torch.full((12, 16), 5.0, device=dev)
        writes(dev)[name](t)
        assert bool((t != 5.0).any())


def test_read_tensors_keep_their_version(dev):
    from weight_communication_gb300 import embedding, fp8, gradnorm
    table, ids = torch.ones(9, 16, device=dev), torch.arange(9, device=dev)
    before = table._version, ids._version
    out = embedding.lookup(table, ids)
    embedding.grad(table, ids, 9)
    fp8.quantize(table, columns=True)
    gradnorm.norm([table])
    gradnorm.clip([table], 1.0, out=[out])
    assert (table._version, ids._version) == before


def test_load_changes_the_codes(dev):
    from weight_communication_gb300 import fp8
    w = torch.ones(130, 40, device=dev)
    lin = fp8.Fp8Linear(w)
    codes = lin.w.codes
    before = codes._version
    lin.load(w)
    assert codes._version > before


def test_a_gradient_that_ends_is_told_of(dev):
    from weight_communication_gb300 import embedding, fp8
    table, ids = torch.ones(9, 16, device=dev, requires_grad=True), torch.arange(9, device=dev)
    lin = fp8.Fp8Linear(torch.ones(24, 16, device=dev, requires_grad=True))
    for call, name in ((lambda: embedding.lookup(table, ids), "lookup"),
                       (lambda: embedding.grad(table, ids, 9), "grad"),
                       (lambda: fp8.quantize(table), "quantize"), (lambda: lin.forward(table), "quantize")):
        with pytest.warns(UserWarning, match=f"{name} stands outside autograd"):
            assert not getattr(call(), "requires_grad", False)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                call()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        # a weight is kept in 8 bits beside the tensor that requires a gradient
        lin.load(torch.ones(24, 16, device=dev, requires_grad=True))
        fp8.quantize_weight(table)
        embedding.lookup(table.detach(), ids)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning, match="outside autograd"):
            embedding.lookup(table, ids)
