"""Embedding rows that start on any element: every remainder of the row
distances by 16 bytes, lookups and gradients, with guards between the rows.
Lookups round once, so they equal the definition; gradients are sums of small
whole numbers, which are exact."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from weight_communication_gb300 import embedding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [129, 255, 1024, 1030, 2045])
@pytest.mark.parametrize("pad_table,pad_out", [(0, 0), (1, 0), (0, 1), (3, 2), (2, 7), (5, 6), (7, 3), (4, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_lookup_rows(dev, D, pad_table, pad_out, dtype, scale):
    g = torch.Generator(device=dev)
    g.manual_seed(D + 10 * pad_table + 100 * pad_out)
    V, n, first = 53, 301, 7
    flat = torch.full((V * (D + pad_table),), float("nan"), dtype=dtype, device=dev)
    table = flat.view(V, D + pad_table)[:, :D]
    table.copy_(torch.randn(V, D, generator=g, device=dev))
    if pad_table == 0:
        table = flat.view(V, D)
    ids = torch.randint(0, V + 2 * first, (n,), generator=g, device=dev)
    ids[:3] = torch.tensor([first + V - 1, -1, first], device=dev)  # the last row, padding, the first
    wide = torch.full((n, D + pad_out), 5.0, dtype=dtype, device=dev)
    out = wide[:, :D]
    embedding.lookup(table, ids, scale=scale, first_row=first, out=out)
    row = ids - first
    live = (row >= 0) & (row < V)
    want = table[row.clamp(0, V - 1)].float() * torch.tensor(scale, dtype=torch.float32, device=dev)
    want = torch.where(live[:, None], want, torch.zeros_like(want)).to(dtype)
    assert torch.equal(out, want)
    assert bool((wide[:, D:] == 5.0).all())


@pytest.mark.parametrize("D,pad", [(129, 0), (1649, 0), (1649, 1), (1001, 2), (8, 3), (3, 0), (1, 0), (5, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_zero_rows(dev, D, pad, dtype):
    g = torch.Generator(device=dev)
    g.manual_seed(D + pad)
    V, n = 997, 60
    dy = torch.randint(-2, 3, (n, D), generator=g, device=dev).to(dtype)
    ids = torch.randint(0, V, (n,), generator=g, device=dev)
    wide = torch.full((V, D + pad), 5.0, dtype=dtype, device=dev)
    got = embedding.grad(dy, ids, V, out=wide[:, :D])
    want = torch.zeros(V, D, device=dev).index_add_(0, ids, dy.float()).to(dtype)
    assert torch.equal(got, want)
    assert bool((wide[:, D:] == 5.0).all())
