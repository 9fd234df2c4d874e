"""Lookups of many tokens whose rows start on any element (2^18 values and
more, where they are read in chunks), against the definition."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from weight_communication_gb300 import embedding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,D,pad", [(3000, 129, 0), (2033, 129, 0), (2032, 129, 0), (3000, 255, 1), (1501, 1001, 2),
                                     (1200, 1030, 0), (700, 2045, 3), (263000, 1, 0), (40000, 127, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_many_tokens(dev, n, D, pad, dtype, id_type):
    g = torch.Generator(device=dev)
    g.manual_seed(n + D)
    V, first = 211, 40
    table = torch.randn(V, D + pad, generator=g, device=dev).to(dtype)[:, :D]
    ids = torch.randint(-3, V + 2 * first, (n,), generator=g, device=dev).to(id_type)
    ids[0], ids[-1] = first + V - 1, first + V - 1  # the table's last row, first and last
    wide = torch.full((n, D + 1), 5.0, dtype=dtype, device=dev)
    for out in (torch.empty(n, D, dtype=dtype, device=dev), wide[:, :D]):
        for scale in (1.0, 45.25):
            embedding.lookup(table, ids, scale=scale, first_row=first, out=out)
            row = ids.long() - first
            live = (row >= 0) & (row < V)
            want = table[row.clamp(0, V - 1)].float() * scale
            assert torch.equal(out, torch.where(live[:, None], want, torch.zeros_like(want)).to(dtype))
    assert bool((wide[:, D] == 5.0).all())
