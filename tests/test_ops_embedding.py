"""Embedding lookup and its gradient on the GPU.

The lookup is one fp32 product and one rounding: equal bits to the same in
torch.  The gradient of a row with c tokens is a sum of c fp32 values in some
fixed order (at most c - 1 roundings of partial sums, each bounded by the sum
of magnitudes), one product with the scale and, when adding, one more sum:
(c + 3) u of the magnitudes, u = 2^-24, and one part in 2^8 (bf16 keeps 8 bits) of the result for
bf16 outputs.
"""
import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


def zipf(n, V, g, first=0, outside=0.1, dtype=torch.int64):
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * torch.log(torch.tensor(V + 1.0, dtype=torch.float64, device="cuda"))).long()
           - 1).clamp(0, V - 1) + first
    r = torch.rand(n, generator=g, device="cuda")
    ids = torch.where(r < outside / 2, torch.full_like(ids, -1), ids)
    ids = torch.where(r > 1 - outside / 2, torch.full_like(ids, first + V), ids)
    return ids.to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def exact_grad(dy, ids, V, scale, first, before=None):
    """(gradient, magnitudes, tokens per row) in 64 bits."""
    row = ids.reshape(-1).long() - first
    live = ((row >= 0) & (row < V)).nonzero()[:, 0]
    d = dy.reshape(row.numel(), dy.shape[-1]).double()[live] * scale
    out = torch.zeros(V, dy.shape[-1], dtype=torch.float64, device=dy.device)
    mag, cnt = out.clone(), torch.zeros(V, dtype=torch.float64, device=dy.device)
    out.index_add_(0, row[live], d)
    mag.index_add_(0, row[live], d.abs())
    cnt.index_add_(0, row[live], torch.ones(live.numel(), dtype=torch.float64, device=dy.device))
    if before is not None:
        out, mag = out + before.double(), mag + before.double().abs()
    return out, mag, cnt


def check_grad(got, dy, ids, V, scale, first, before=None):
    want, mag, cnt = exact_grad(dy, ids, V, scale, first, before)
    tol = (cnt[:, None] + 3) * U * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((got.double() - want).abs() <= tol).all())
    if before is not None:
        idle = cnt == 0
        assert torch.equal(got[idle], before[idle])


@pytest.mark.parametrize("V,D,n", [(1, 1, 1), (5, 3, 40), (1000, 64, 17), (321, 100, 1), (97, 129, 300),
                                   (4000, 2048, 700), (33, 4098, 50), (2000, 8, 5000), (10, 20, 0)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_lookup(dev, V, D, n, dtype, id_type):
    from weight_communication_gb300 import embedding
    g = gen(21)
    table = torch.randn(V, D, generator=g, device=dev).to(dtype)
    for first, scale in ((0, 1.0), (3 * V, 1.7)):
        ids = zipf(n, V, g, first, 0.3, id_type)
        row = ids.long() - first
        live = (row >= 0) & (row < V)
        want = (table[row.clamp(0, V - 1)].float() * scale).to(dtype)
        want = torch.where(live[:, None], want, torch.zeros_like(want))
        assert torch.equal(embedding.lookup(table, ids, scale, first), want)


def test_lookup_shapes_strides_and_guards(dev):
    """Ids of any shape; table and output rows further apart than D."""
    from weight_communication_gb300 import embedding
    g = gen(22)
    wide = torch.randn(50, 48, generator=g, device=dev)
    table = wide[:, :24]
    ids = torch.randint(0, 50, (3, 4, 5), generator=g, device=dev)
    assert torch.equal(embedding.lookup(table, ids), table[ids])
    out = torch.full((60, 40), -5.0, device=dev)
    embedding.lookup(table, ids, 2.0, out=out[:, :24])
    assert torch.equal(out[:, :24], table[ids.view(-1)] * 2.0)
    assert bool((out[:, 24:] == -5.0).all())


def test_extreme_ids(dev):
    from weight_communication_gb300 import embedding
    table = torch.ones(8, 16, device=dev)
    ids = torch.tensor([-2 ** 63, 2 ** 63 - 1, -1, 8 + 2 ** 40, 2 ** 40 + 7, 2 ** 40], device=dev)
    out = embedding.lookup(table, ids, first_row=2 ** 40)
    assert out[:, 0].tolist() == [0.0, 0.0, 0.0, 0.0, 1.0, 1.0]
    d = embedding.grad(torch.ones(6, 16, device=dev), ids, 8, first_row=2 ** 40)
    assert d[:, 3].tolist() == [1.0] + [0.0] * 6 + [1.0]


@pytest.mark.parametrize("V,D,n", [(1, 1, 1), (1, 8, 5000), (5, 3, 40), (1000, 64, 17), (97, 129, 300),
                                   (4001, 2048, 3000), (33, 4098, 500), (20_000, 24, 9000), (12, 7, 0),
                                   (400_000, 9, 2000), (700, 4096, 64)])
@pytest.mark.parametrize("dy_type", TYPES)
@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad(dev, V, D, n, dy_type, out_type, accumulate):
    from weight_communication_gb300 import embedding
    g = gen(23)
    dy = torch.randn(n, D, generator=g, device=dev).to(dy_type)
    first = 2 * V if n % 2 else 0
    ids = zipf(n, V, g, first, 0.2, torch.int32 if n % 3 else torch.int64)
    before = torch.randn(V, D, generator=g, device=dev).to(out_type) if accumulate else None
    out = before.clone() if accumulate else torch.full((V, D), 9.0, dtype=out_type, device=dev)
    got = embedding.grad(dy, ids, V, 1.5, first, out=out, accumulate=accumulate)
    assert got is out
    check_grad(got, dy, ids, V, 1.5, first, before)


@pytest.mark.parametrize("n", [2, 600, 5000, 40_000])
def test_grad_of_one_hot_row(dev, n):
    """All tokens the same: one row spread over every worker."""
    from weight_communication_gb300 import embedding
    dy = torch.randn(n, 264, generator=gen(24), device=dev)
    ids = torch.full((n,), 77, device=dev)
    got = embedding.grad(dy, ids, 100)
    check_grad(got, dy, ids, 100, 1.0, 0)
    assert bool((got[:77] == 0).all()) and bool((got[78:] == 0).all())


def test_grad_without_any_token(dev):
    from weight_communication_gb300 import embedding
    dy = torch.ones(10, 12, device=dev)
    ids = torch.full((10,), -1, device=dev)
    out = torch.full((6, 12), 4.0, device=dev)
    embedding.grad(dy, ids, 6, out=out, accumulate=True)
    assert bool((out == 4.0).all())
    embedding.grad(dy, ids, 6, out=out)
    assert bool((out == 0.0).all())


def test_grad_skips_values_of_tokens_outside(dev):
    """dy of padding tokens may hold anything, NaN included."""
    from weight_communication_gb300 import embedding
    dy = torch.ones(100, 32, device=dev)
    ids = torch.arange(100, device=dev) % 10
    dy[ids == 3] = float("nan")
    ids[ids == 3] = -1
    got = embedding.grad(dy, ids, 10)
    assert got[:, 0].tolist() == [10.0 if v != 3 else 0.0 for v in range(10)]


def test_grad_strides_and_guards(dev):
    from weight_communication_gb300 import embedding
    g = gen(25)
    dy = torch.randn(70, 80, generator=g, device=dev)[:, :36]
    ids = torch.randint(0, 9, (70,), generator=g, device=dev)
    out = torch.full((9, 60), -5.0, device=dev)
    embedding.grad(dy, ids, 9, out=out[:, :36])
    check_grad(out[:, :36], dy, ids, 9, 1.0, 0)
    assert bool((out[:, 36:] == -5.0).all())


def test_grad_is_the_same_every_run(dev):
    from weight_communication_gb300 import embedding
    g = gen(26)
    dy = torch.randn(20_000, 512, generator=g, device=dev).bfloat16()
    ids = zipf(20_000, 3000, g)
    first = embedding.grad(dy, ids, 3000, out_dtype=torch.float32)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(4):
        again = embedding.grad(dy, ids, 3000, out_dtype=torch.float32, stream=s)
        s.synchronize()
        assert torch.equal(again, first)


def test_grad_against_differences(dev):
    """d(sum of out * dy)/d table by differences of the lookup, which is linear
    in the table: exact on small multiples of 1/64."""
    from weight_communication_gb300 import embedding
    g = gen(27)
    V, D, n = 11, 10, 60
    table = torch.randint(-64, 65, (V, D), generator=g, device=dev).float() / 64
    dy = torch.randint(-64, 65, (n, D), generator=g, device=dev).float() / 64
    ids = zipf(n, V, g, 0, 0.2)

    def loss(t):
        return float((embedding.lookup(t, ids, 0.5).double() * dy.double()).sum())

    got = embedding.grad(dy, ids, V, 0.5)
    for v in range(V):
        for c in (0, D // 2, D - 1):
            up, down = table.clone(), table.clone()
            up[v, c] += 1.0
            down[v, c] -= 1.0
            assert float(got[v, c]) == (loss(up) - loss(down)) / 2


def test_offsets_beyond_32_bits(dev):
    """Tables and outputs of more than 2^32 values (bf16)."""
    from weight_communication_gb300 import embedding
    V, D = 1 << 21, 2056
    table = torch.zeros(V, D, dtype=torch.bfloat16, device=dev)
    rows = torch.tensor([0, 1 << 20, (1 << 20) + 1, V - 1], device=dev)
    table[rows] = torch.arange(1.0, 5.0, device=dev).bfloat16()[:, None]
    out = embedding.lookup(table, rows)
    assert out[:, 0].tolist() == [1.0, 2.0, 3.0, 4.0] and out[:, -1].tolist() == [1.0, 2.0, 3.0, 4.0]
    embedding.grad(out, rows, V, out=table)
    assert torch.equal(table[rows], out)
    assert int((table[:, 0] != 0).sum()) == 4 and int((table[:, -1] != 0).sum()) == 4
