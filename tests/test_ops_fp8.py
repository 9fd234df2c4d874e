"""8-bit block-scaled quantization and products on the GPU.

Quantization: equal codes and scales to the definition, computed here in
numpy by binary32 divisions and products and the e4m3 grid.

Products: the operands' codes and scales are exact inputs, so only the sums
round.  Within a block of 128 the tensor core adds 128 exact products; nothing
is assumed of it but that an addition loses at most 2^-23 of the largest
magnitude, 128 * 2u (u = 2^-24).  Outside, one product of the two scales, and
one fma per block: (256 + blocks + 4) u of the sum of magnitudes, plus half of
2^-8 of the result for bf16 outputs.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def values(t):
    """What an Fp8Tensor stands for, in 64 bits."""
    s = t.scales.double().repeat_interleave(128, 0)[:t.cols].t()
    s = s.repeat_interleave(t.block_rows, 0)[:t.rows]
    return t.codes[:, :t.cols].double() * s


def check(got, a, b, before=None):
    A, B = values(a), values(b)
    want, mag = A @ B.t(), A.abs() @ B.abs().t()
    if before is not None:
        want, mag = want + before.double(), mag + before.double().abs()
    tol = (256 + -(-a.cols // 128) + 4) * U * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((got.double() - want).abs() <= tol).all())


# ---------------------------------------------------------------------------
# quantization
# ---------------------------------------------------------------------------

def e4m3(v):
    """Nearest e4m3 value of binary32 values in [-448, 448], ties to even."""
    v = v.astype(np.float64)
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(v / step) * step


def reference(x, square):
    """(codes, scales) of x [R, C] fp32 by blocks of 128 columns."""
    R, C = x.shape
    cb = -(-C // 128)
    codes = np.zeros((R, C))
    step = 128 if square else 1
    scales = np.zeros((cb, -(-R // step)), np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for b in range(cb):
            for r in range(0, R, step):
                part = x[r:r + step, b * 128:(b + 1) * 128]
                m = np.abs(part).max()
                if not np.isfinite(part).all():
                    scales[b, r // step] = np.nan
                elif m >= np.float32(448 * 2.0 ** -126):
                    scales[b, r // step] = m / np.float32(448)
                    codes[r:r + step, b * 128:(b + 1) * 128] = e4m3(part * (np.float32(448) / m))
    return codes, scales


def check_quant(t, x, square):
    codes, scales = reference(x.float().cpu().numpy(), square)
    np.testing.assert_array_equal(t.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(t.codes[:, :t.cols].float().cpu().numpy().astype(np.float64), codes)
    assert bool((t.codes[:, t.cols:].float() == 0).all())


@pytest.mark.parametrize("M,K", [(1, 1), (1, 300), (5, 128), (128, 128), (130, 257), (300, 16), (17, 1000),
                                 (129, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("square", [False, True])
def test_quantize(dev, M, K, dtype, square):
    from weight_communication_gb300 import fp8
    x = torch.randn(M, K, generator=gen(31), device=dev)
    x = (x * torch.exp(3 * torch.randn(M, 1, generator=gen(32), device=dev))).to(dtype)
    f = fp8.quantize_weight if square else fp8.quantize
    q, qt = f(x, columns=True)
    check_quant(q, x, square)
    check_quant(qt, x.t(), square)
    only, none = f(x)
    assert none is None and torch.equal(only.codes.view(torch.uint8), q.codes.view(torch.uint8))
    none, only = f(x, rows=False, columns=True)
    assert none is None and torch.equal(only.codes.view(torch.uint8), qt.codes.view(torch.uint8))


def test_quantize_edge_blocks(dev):
    """Zero, subnormal, threshold, tiny and huge blocks; exact ties."""
    from weight_communication_gb300 import fp8
    x = torch.zeros(12, 200, device=dev)
    x[1, :3] = torch.tensor([1e-45, -1e-39, 2e-38], device=dev)
    x[2, 5] = 448 * 2.0 ** -126
    x[3, 5] = float(np.nextafter(np.float32(448 * 2.0 ** -126), np.float32(0)))
    x[4, :2] = torch.tensor([3.4e38, -1e38], device=dev)
    x[5, :4] = torch.tensor([448.0, 17.0, 19.0, -2.0 ** -10], device=dev)      # ties of the grid
    x[6] = -0.0
    x[7, 130:] = 5.0
    x[8] = torch.linspace(-1, 1, 200, device=dev)
    q, qt = fp8.quantize(x, columns=True)
    check_quant(q, x, False)
    check_quant(qt, x.t(), False)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_values_that_are_not_finite(dev, bad):
    """Their block gets scale NaN and codes 0; the outputs it enters are NaN
    and no others."""
    from weight_communication_gb300 import fp8
    x = torch.randn(40, 300, generator=gen(33), device=dev).bfloat16()
    x[7, 140] = bad
    q, qt = fp8.quantize(x, columns=True)
    check_quant(q, x, False)
    check_quant(qt, x.t(), False)
    w, _ = fp8.quantize_weight(torch.randn(60, 300, generator=gen(34), device=dev))
    y = fp8.matmul(q, w)
    assert bool(y[7].isnan().all()) and not bool(y[:7].isnan().any()) and not bool(y[8:].isnan().any())


def test_quantize_strided_and_guarded(dev):
    from weight_communication_gb300 import binding, fp8
    wide = torch.randn(70, 400, generator=gen(35), device=dev).bfloat16()
    x = wide[:, :250]
    q, _ = fp8.quantize(x)
    check_quant(q, x, False)
    codes = torch.full((70, 304), 1.0, device=dev).to(torch.float8_e4m3fn)
    scales = torch.full((2, 80), -1.0, device=dev)
    binding.fp8_quant(x, codes, scales)
    assert torch.equal(codes[:, :250].float(), q.codes[:, :250].float())
    assert bool((codes[:, 250:256].float() == 0).all()) and bool((codes[:, 256:].float() == 1).all())
    assert torch.equal(scales[:, :70], q.scales) and bool((scales[:, 70:] == -1).all())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 300, 2048), (3, 129, 100), (16, 128, 128), (17, 500, 384), (32, 1003, 1501),
          (33, 64, 4096), (64, 257, 640), (65, 300, 200), (128, 256, 128), (129, 255, 129),
          (200, 1000, 3000), (333, 1003, 1501), (1000, 700, 128), (2049, 2500, 300), (128, 5000, 64),
          (2600, 3000, 1000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("a_square,b_square", [(False, True), (False, False), (True, True), (True, False)])
def test_matmul(dev, M, N, K, a_square, b_square):
    from weight_communication_gb300 import binding, fp8
    x = torch.randn(M, K, generator=gen(41), device=dev)
    w = torch.randn(N, K, generator=gen(42), device=dev)
    a, _ = (fp8.quantize_weight if a_square else fp8.quantize)(x)
    b, _ = (fp8.quantize_weight if b_square else fp8.quantize)(w)
    for dtype in (torch.float32, torch.bfloat16):
        check(fp8.matmul(a, b, out_dtype=dtype), a, b)
    before = torch.randn(M, N, generator=gen(43), device=dev)
    check(fp8.matmul(a, b, out=before.clone(), accumulate=True), a, b, before)
    assert binding.wait_timeouts() == 0


@pytest.mark.parametrize("M,N", [(5, 70), (40, 130), (100, 90), (200, 1000), (3000, 2900)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_into_a_wider_buffer(dev, M, N, dtype):
    """Output rows further apart than N, odd distances included; the values
    between them stay."""
    from weight_communication_gb300 import fp8
    a, _ = fp8.quantize(torch.randn(M, 260, generator=gen(44), device=dev))
    b, _ = fp8.quantize_weight(torch.randn(N, 260, generator=gen(45), device=dev))
    for extra in (1, 8, 40):
        out = torch.full((M, N + extra), -3.0, dtype=dtype, device=dev)
        check(fp8.matmul(a, b, out=out[:, :N]), a, b)
        assert bool((out[:, N:] == -3.0).all())


def test_matmul_of_views(dev):
    """Operands that are some rows, or some blocks of columns, of others."""
    from weight_communication_gb300 import fp8
    a, _ = fp8.quantize(torch.randn(400, 1024, generator=gen(46), device=dev))
    b, _ = fp8.quantize(torch.randn(300, 1024, generator=gen(47), device=dev))
    rows = fp8.Fp8Tensor(a.codes[16:200], a.scales[:, 16:200].contiguous(), 184, 1024)
    check(fp8.matmul(rows, b, out_dtype=torch.float32), rows, b)
    ac = fp8.Fp8Tensor(a.codes[:, 256:768], a.scales[2:6], 400, 512)
    bc = fp8.Fp8Tensor(b.codes[:, 256:768], b.scales[2:6], 300, 512)
    check(fp8.matmul(ac, bc, out_dtype=torch.float32), ac, bc)


def test_matmul_with_nothing_to_sum(dev):
    from weight_communication_gb300 import fp8
    a = fp8.Fp8Tensor.empty(70, 0)
    b = fp8.Fp8Tensor.empty(90, 0)
    out = torch.full((70, 90), 5.0, device=dev)
    fp8.matmul(a, b, out=out, accumulate=True)
    assert bool((out == 5.0).all())
    fp8.matmul(a, b, out=out)
    assert bool((out == 0.0).all())
    c, _ = fp8.quantize(torch.empty(0, 64, device=dev))
    d, _ = fp8.quantize(torch.ones(5, 64, device=dev))
    assert fp8.matmul(c, d).shape == (0, 5) and fp8.matmul(d, c).shape == (5, 0)


def test_matmul_same_bits_every_run_and_on_another_stream(dev):
    from weight_communication_gb300 import fp8
    a, _ = fp8.quantize(torch.randn(1500, 2000, generator=gen(48), device=dev))
    b, _ = fp8.quantize(torch.randn(1700, 2000, generator=gen(49), device=dev))
    for rows in (7, 50, 1500):
        p = fp8.Fp8Tensor(a.codes[:rows], a.scales[:, :rows].contiguous(), rows, 2000)
        first = fp8.matmul(p, b, out_dtype=torch.float32)
        s = torch.cuda.Stream(dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        for _ in range(3):
            again = fp8.matmul(p, b, out_dtype=torch.float32, stream=s)
            s.synchronize()
            assert torch.equal(again, first)


def test_offsets_beyond_32_bits(dev):
    """An output of more than 2^32 values, and operands of 2^31 rows x K / 128."""
    from weight_communication_gb300 import fp8
    M, N = 70_000, 62_000
    a, _ = fp8.quantize(torch.randn(M, 16, generator=gen(50), device=dev))
    b, _ = fp8.quantize(torch.randn(N, 16, generator=gen(51), device=dev))
    y = fp8.matmul(a, b)
    A, B = values(a), values(b)
    for rows in (slice(0, 100), slice(34_600, 34_800), slice(M - 100, M)):
        want, mag = A[rows] @ B.t(), A[rows].abs() @ B.abs().t()
        tol = 261 * U * mag
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
        assert bool(((y[rows].double() - want).abs() <= tol).all())


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (100, 300, 200), (777, 1111, 555), (513, 256, 1024)])
def test_layer_forward_and_backward(dev, M, N, K):
    """y, dx and dw against 64-bit products of what was quantized."""
    from weight_communication_gb300 import fp8
    x = torch.randn(M, K, generator=gen(61), device=dev).bfloat16()
    w = (0.02 * torch.randn(N, K, generator=gen(62), device=dev)).bfloat16()
    dy = (1e-3 * torch.randn(M, N, generator=gen(63), device=dev)).bfloat16()
    lin = fp8.Fp8Linear(w)
    y, saved = lin.forward(x, save=True)
    assert torch.equal(lin.forward(x), y)
    dx, dw = lin.backward(dy, saved)
    xq, xt = fp8.quantize(x, columns=True)
    dq, dt = fp8.quantize(dy, columns=True)
    check(y, xq, lin.w)
    check(dx, dq, lin.wt)
    check(dw, dt, xt)
    assert y.dtype == dx.dtype == torch.bfloat16 and dw.dtype == torch.float32
    more = dw.clone()
    _, same = lin.backward(dy, saved, dw=more, accumulate=True)
    assert same is more
    check(more, dt, xt, dw)
    lin.load(2 * w)
    assert torch.equal(lin.forward(x).float(), 2 * y.float())


def test_layer_against_differences(dev):
    """Gradients by differences of the forward pass, on inputs that 8 bits hold
    exactly (multiples of 8 up to 64, 448 on the diagonals so that every
    block's scale is 1): the loss sum(y * dy) is linear in x and in w, so the
    differences are exact."""
    from weight_communication_gb300 import fp8
    n = 40
    grid = torch.tensor([-64.0, -48.0, -16.0, 0.0, 16.0, 32.0, 56.0], device=dev)

    def draw(seed):
        t = grid[torch.randint(0, 7, (n, n), generator=gen(seed), device=dev)]
        t.fill_diagonal_(448.0)
        return t

    x, w, dy = draw(71), draw(72), draw(73)

    def loss(x, w):
        y = fp8.Fp8Linear(w, training=False).forward(x, out_dtype=torch.float32)
        return float((y.double() * dy.double()).sum())

    lin = fp8.Fp8Linear(w)
    _, saved = lin.forward(x, save=True)
    dx, dw = lin.backward(dy, saved, dx_dtype=torch.float32)
    for r, c in ((0, 1), (5, 17), (39, 2), (20, 38)):
        for t, got in ((x, dx), (w, dw)):
            ends = []
            for h in (8.0, -8.0):
                moved = t.clone()
                moved[r, c] = 48.0 + h
                ends.append(loss(moved, w) if t is x else loss(x, moved))
            assert float(got[r, c]) == (ends[0] - ends[1]) / 16.0
