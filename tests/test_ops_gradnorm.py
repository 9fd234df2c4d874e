"""Gradient norm and clipping on the GPU against 64-bit sums.

Tolerances, from the kernels' arithmetic (u = 2^-24, half the spacing of
binary32 at 1): 32 squares are summed in fp32 in chains of 4 fused
multiply-adds and 3 levels of adds, at most 7 roundings, and everything above
that is as good as exact, so the sum of squares is within 7u, its root within
3.5u, and the stored norm within 5u with its own rounding.  The coefficient
inherits the root's error and one rounding (5u), a product one more (6u);
bf16 outputs add one part in 2^8 (bf16 keeps 8 bits).
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def exact_norm(tensors) -> float:
    return math.sqrt(math.fsum(float(np.dot(a, a)) for a in
                               (t.detach().double().cpu().numpy().ravel() for t in tensors)))


def check_clip(before, after, stats, max_norm, eps=1e-6):
    n = exact_norm(before)
    norm, coef = float(stats[0]), float(stats[1])
    assert abs(norm - n) <= 5 * U * n
    want = min(1.0, max_norm / (n + eps)) if n + eps > 0 else 1.0
    assert abs(coef - want) <= 5 * U * want
    for b, a in zip(before, after):
        x = b.double() * want
        tol = x.abs() * (6 * U + (2.0 ** -8 if a.dtype == torch.bfloat16 else 0.0)) + 1e-40
        assert bool(((a.double() - x).abs() <= tol).all())


def draw(sizes, dtypes, seed, sigma=1e-3, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device=device) * sigma).to(dt)
            for n, dt in zip(sizes, dtypes)]


SIZES = [[1], [7], [8], [31, 1, 8192], [8191, 8193, 16385, 3], [100_000, 1, 0, 5], [1 << 20],
         [12_289 * 5, 33, 65_536], [300] * 65, [17] * 64]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("types", ["bf16", "f32", "mixed"])
def test_norm_and_clip_into_other_buffers(dev, sizes, types):
    from weight_communication_gb300 import gradnorm
    pick = {"bf16": [torch.bfloat16], "f32": [torch.float32],
            "mixed": [torch.bfloat16, torch.float32]}[types]
    grads = draw(sizes, [pick[i % len(pick)] for i in range(len(sizes))], 11)
    n = exact_norm(grads)
    assert abs(float(gradnorm.norm(grads)) - n) <= 5 * U * n
    for out_type in (torch.float32, torch.bfloat16):
        for bound in (0.3 * n, 2.0 * n):
            out = [torch.full(g.shape, 9.0, dtype=out_type, device=dev) for g in grads]
            stats = gradnorm.clip(grads, bound, out=out)
            check_clip(grads, out, stats, bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place(dev, dtype):
    from weight_communication_gb300 import gradnorm
    grads = draw([9001, 5, 70_000], [dtype] * 3, 12)
    before = [g.clone() for g in grads]
    n = exact_norm(before)
    stats = gradnorm.clip(grads, 10.0 * n)          # within the bound: untouched
    assert float(stats[1]) == 1.0
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    stats = gradnorm.clip(grads, 0.5 * n)
    check_clip(before, grads, stats, 0.5 * n)


@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("out_shift", [0, 1, 2])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32])
def test_any_offset_into_a_flat_buffer(dev, shift, out_shift, src, dst):
    """Views that start anywhere; the values around them stay as they are."""
    from weight_communication_gb300 import gradnorm
    sizes = [3, 8200, 1, 0, 20_001]
    flat = draw([sum(sizes) + 32], [src], 13)[0]
    guard = torch.full((sum(sizes) + 32,), -7.0, dtype=dst, device=dev)
    grads, outs, a, b = [], [], shift, out_shift
    for n in sizes:
        grads.append(flat[a:a + n])
        outs.append(guard[b:b + n])
        a, b = a + n, b + n
    n = exact_norm(grads)
    stats = gradnorm.clip(grads, 0.25 * n, out=outs)
    check_clip(grads, outs, stats, 0.25 * n)
    assert bool((guard[:out_shift] == -7.0).all()) and bool((guard[b:] == -7.0).all())


def test_more_tensors_than_one_launch_takes(dev):
    from weight_communication_gb300 import gradnorm
    grads = draw([1 + (7 * i) % 97 for i in range(2500)], [torch.float32, torch.bfloat16] * 1250, 14)
    n = exact_norm(grads)
    assert abs(float(gradnorm.norm(grads)) - n) <= 5 * U * n
    before = [g.clone() for g in grads]
    stats = gradnorm.clip(grads, 0.1 * n)
    check_clip(before, grads, stats, 0.1 * n)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-25, 1e-38, 1e-44])
def test_values_whose_squares_leave_binary32(dev, value):
    """Finite gradients have a finite norm, tiny ones do not vanish."""
    from weight_communication_gb300 import gradnorm
    x = torch.full((10_007,), value, device=dev)
    x[::3] = 0.0
    y = torch.full((5,), value, dtype=torch.bfloat16, device=dev)
    n = exact_norm([x, y])
    got = float(gradnorm.norm([x, y]))
    if n > 3.4e38:
        assert math.isinf(got)
    else:
        assert abs(got - n) <= 5 * U * n + 1.5e-45


def test_zero_and_empty(dev):
    from weight_communication_gb300 import gradnorm
    z = torch.zeros(5000, device=dev)
    e = torch.empty(0, device=dev, dtype=torch.bfloat16)
    stats = gradnorm.clip([z, e], 1.0)
    assert stats.tolist() == [0.0, 1.0]
    assert gradnorm.clip([e], 1.0).tolist() == [0.0, 1.0]
    assert gradnorm.norm([e]).tolist() == [0.0]
    assert bool((z == 0).all())


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_values_that_are_not_finite(dev, bad):
    """An infinite norm gives coefficient 0 (and 0 * inf = NaN there), one
    that is not a number gives NaN everywhere."""
    from weight_communication_gb300 import gradnorm
    x = torch.ones(20_000, device=dev)
    x[12_345] = bad
    out = torch.empty_like(x)
    stats = gradnorm.clip([x], 1.0, out=[out]).tolist()
    if math.isinf(bad):
        assert stats == [math.inf, 0.0]
        assert math.isnan(float(out[12_345])) and float(out.nan_to_num(0.0).abs().max()) == 0.0
    else:
        assert math.isnan(stats[0]) and math.isnan(stats[1]) and bool(out.isnan().all())


def test_same_bits_every_run_and_on_another_stream(dev):
    from weight_communication_gb300 import gradnorm
    grads = gradnorm.TensorList(draw([1_000_003, 77, 250_000], [torch.bfloat16] * 3, 15))
    first = gradnorm.norm(grads).clone()
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(5):
        out = [torch.empty_like(t) for t in grads.tensors]
        again = gradnorm.clip(grads, 0.2, out=out, stream=s)
        s.synchronize()
        assert torch.equal(again[:1], first)


def test_capture_in_a_graph(dev):
    from weight_communication_gb300 import gradnorm
    grads = gradnorm.TensorList(draw([50_000, 9], [torch.float32] * 2, 16))
    out = gradnorm.TensorList([torch.empty_like(t) for t in grads.tensors])
    want = gradnorm.clip(grads, 0.01, out=out).clone()
    want_out = [t.clone() for t in out.tensors]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stats = gradnorm.clip(grads, 0.01, out=out)
    for t in out.tensors:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(stats, want)
    assert all(torch.equal(a, b) for a, b in zip(out.tensors, want_out))


def test_large_list(dev):
    """A tensor with more values than 32 bits index (bf16, 8.6 GB)."""
    from weight_communication_gb300 import gradnorm
    n = (1 << 32) + 12_345
    x = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    at = torch.tensor([0, 5, (1 << 31) + 1, (1 << 32) - 1, 1 << 32, n - 1], device=dev)
    x[at] = 3.0
    norm = math.sqrt(6 * 9.0)
    stats = gradnorm.clip([x], 0.5 * norm)
    assert abs(float(stats[0]) - norm) <= 5 * U * norm
    assert x[at].tolist() == [1.5] * 6
    assert int((x != 0).sum()) == 6
