"""Cross entropy over a vocabulary without its logits, against 64-bit formulas."""
import pytest
import torch

from gpu_util import dev  # noqa: F401
from layers_util import HALF_STEP, TINY, ULP, close, strided

pytestmark = pytest.mark.gpu


def inputs(dev, T, V, D, wide=True, padding=True, seed=0, sigma=None):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device=dev) * (sigma or D ** -0.5)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device=dev)
    x = torch.randn(T, D, generator=g, device=dev)
    x += torch.rand(T, 1, generator=g, device=dev) * 6 * w[y].float() / max(1e-6, float(w.float().square().sum(1).mean()))
    if padding:
        y[::5] = -100
        y[3::7] = V
    return x.bfloat16(), w, y if wide else y.int()


def reference(x, w, y, dlosses):
    """(values, what each may be off by) of losses, lse, dx, dw."""
    T, D = x.shape
    V = w.shape[0]
    xd, wd = x.double(), w.double()
    s = xd @ wd.t()
    lse = torch.logsumexp(s, 1)
    live = (y >= 0) & (y < V)
    at = torch.where(live, y.long(), 0)
    sy = s.gather(1, at[:, None])[:, 0]
    losses = torch.where(live, lse - sy, 0.0)
    # a logit: every step of the sum may lose an ulp of what it has summed
    off_s = (D + 16) * 2 * ULP * (xd.abs() @ wd.abs().t()).amax(1)
    off_lse = off_s + (lse.abs() + s.abs().amax(1) + 128) * 4 * ULP
    g = torch.where(live, torch.as_tensor(dlosses, device=x.device, dtype=torch.float64).expand(T), 0.0)
    p = torch.exp(s - lse[:, None])
    d = p.clone()
    d.scatter_add_(1, at[:, None], torch.full_like(d[:, :1], -1.0))
    d *= g[:, None]
    # an exponential carries the errors of both logits; then one rounding to bf16
    off_d = g.abs()[:, None] * (p * (off_s + off_lse + (s.abs().amax(1) + lse.abs() + 16) * 4 * ULP)[:, None] + 2 * ULP * p)
    # (an exponential below the smallest normal number, 2^-126, may come as 0)
    off_d = (off_d + HALF_STEP[torch.bfloat16] * d.abs() + g.abs()[:, None] * TINY) * 1.01
    x0 = torch.where(live[:, None], xd, 0.0)
    dx, dw = d @ wd, d.t() @ x0
    off_dx = off_d @ wd.abs() + (V + 16) * 2 * ULP * (d.abs() @ wd.abs())
    off_dw = off_d.t() @ x0.abs() + (T + 16) * 2 * ULP * (d.abs().t() @ x0.abs())
    return (losses, lse, dx, dw), (off_s + off_lse, off_lse, off_dx, off_dw)


def check(x, w, y, dlosses, losses, lse, dx, dw, old=0.0):
    want, off = reference(x, w, y, dlosses)
    V = w.shape[0]
    assert bool((losses[(y < 0) | (y >= V)] == 0).all())
    close(losses, want[0], off[0] + want[0].abs() * 2 * ULP, "losses")
    close(lse, want[1], off[1], "lse")
    if dx is not None:
        assert bool((dx[(y < 0) | (y >= V)] == 0).all())
        close(dx, want[2], off[2] + want[2].abs() * HALF_STEP[dx.dtype] * 1.01 + 1e-37, "dx")
    if dw is not None:
        total = want[3] + old
        close(dw, total, off[3] + total.abs() * HALF_STEP[dw.dtype] * 1.01 + 1e-37, "dw")


SIZES = [(1, 1, 1), (1, 300, 64), (5, 1000, 72), (2, 256, 8), (128, 128, 64), (256, 256, 256), (257, 511, 130),
         (300, 4000, 520), (1, 32000, 512), (64, 5000, 1001), (777, 1003, 333), (1500, 700, 64), (33, 20011, 96),
         (700, 3, 200), (3000, 1000, 512), (1900, 1300, 64), (12, 14000, 72)]


@pytest.mark.parametrize("T,V,D", SIZES)
def test_sizes(dev, T, V, D):
    from weight_communication_gb300 import binding, loss
    for wide in (True, False):
        x, w, y = inputs(dev, T, V, D, wide)
        losses, lse = loss.cross_entropy(x, w, y, save=True)
        torch.cuda.synchronize()
        assert binding.wait_timeouts() == 0
        check(x, w, y, 0.0, losses, lse, None, None)
        assert torch.equal(loss.cross_entropy(x, w, y), losses)
        g = torch.randn(T, device=dev) if wide else 1.0 / T
        dx, dw = loss.cross_entropy_grad(x, w, y, lse, g)
        torch.cuda.synchronize()
        assert binding.wait_timeouts() == 0
        assert dx.dtype == dw.dtype == torch.bfloat16
        check(x, w, y, g, losses, lse, dx, dw)
        again = loss.cross_entropy_grad(x, w, y, lse, g)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("V,D", [(700, 257), (6000, 128), (5001, 1001)])
def test_few_tokens(dev, T, V, D):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, T, V, D, padding=False, seed=T)
    if T > 2:
        y[1] = -1
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    check(x, w, y, 0.0, losses, lse, None, None)
    ws = strided(w, D + 3, 5)
    again, lse2 = loss.cross_entropy(x, ws, y, save=True)
    check(x, w, y, 0.0, again, lse2, None, None)


@pytest.mark.parametrize("T,V,D,ld_x,ld_w,offset", [(70, 333, 64, 72, 80, 0), (70, 333, 64, 65, 64, 0), (70, 333, 64, 64, 67, 3),
                                                    (300, 1000, 200, 208, 200, 1), (300, 1000, 203, 203, 211, 7)])
def test_rows_that_start_anywhere(dev, T, V, D, ld_x, ld_w, offset):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, T, V, D, seed=1)
    xs, ws = strided(x, ld_x, offset), strided(w, ld_w, offset)
    losses, lse = loss.cross_entropy(xs, ws, y, save=True)
    out = strided(torch.zeros_like(w), ld_w + 1, offset)
    before = out._base.clone()
    dx, dw = loss.cross_entropy_grad(xs, ws, y, lse, 0.01, dw=out)
    assert dw is out
    check(x, w, y, 0.01, losses, lse, dx, dw)
    out.copy_(strided(torch.zeros_like(w), ld_w + 1, offset))
    assert torch.equal(out._base, before)     # nothing beside it is written


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,D", [(300, 1000, 256), (90, 517, 131), (2000, 300, 72)])
def test_weight_gradients_and_accumulation(dev, dtype, T, V, D):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, T, V, D, seed=2)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    g = torch.rand(T, device=dev)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, g, dw_dtype=dtype)
    assert dw.dtype == dtype
    check(x, w, y, g, losses, lse, dx, dw)
    old = (torch.randn(V, D, device=dev) * 0.1).to(dtype)
    buf = old.clone()
    dx2, dw2 = loss.cross_entropy_grad(x, w, y, lse, g, dw=buf, accumulate=True)
    assert dw2 is buf and torch.equal(dx2, dx)
    check(x, w, y, g, losses, lse, None, dw2, old.double())
    only, none = loss.cross_entropy_grad(x, w, y, lse, g, needs_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = loss.cross_entropy_grad(x, w, y, lse, g, dw_dtype=dtype, needs_dx=False)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("V,D", [(1, 1), (3, 8), (700, 257), (2000, 64), (5001, 1001), (600, 512), (900, 1024), (20003, 2048),
                                 (700, 4096), (333, 4090), (300, 4104)])
def test_few_tokens_gradients(dev, T, V, D):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, T, V, D, wide=T % 2 == 0, padding=False, seed=T + 20)
    if T > 2:
        y[1] = -1
        x[1] = float("nan")
    _, lse = loss.cross_entropy(x, w, y, save=True)
    g = torch.randn(T, device=dev) if T % 2 else 0.3
    clean = x.clone()
    clean[(y < 0)] = 0
    (_, _, dx0, dw0), (_, _, off_dx, off_dw) = reference(clean, w, y, g)
    if D <= 4096:
        # d is not rounded: a term's bound there without its half step of bf16
        xd, wd = clean.double(), w.double()
        s = xd @ wd.t()
        live = (y >= 0)[:, None]
        p = torch.where(live, torch.exp(s - torch.logsumexp(s, 1)[:, None]), 0.0)
        d = p.clone()
        d.scatter_add_(1, torch.where(y >= 0, y.long(), 0)[:, None], torch.where(live, -1.0, 0.0).double())
        gd = torch.as_tensor(g, device=dev, dtype=torch.float64).expand(T)[:, None].abs()
        rounding = (HALF_STEP[torch.bfloat16] - 4 * ULP) * (gd * d.abs())
        off_dx, off_dw = off_dx - rounding @ wd.abs(), off_dw - rounding.t() @ xd.abs()
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, g)
    assert bool((dx[y < 0] == 0).all())
    close(dx, dx0, off_dx + dx0.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-37, "dx")
    close(dw, dw0, off_dw + dw0.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-37, "dw")
    again = loss.cross_entropy_grad(x, w, y, lse, g)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    only, none = loss.cross_entropy_grad(x, w, y, lse, g, needs_dw=False)
    assert none is None and torch.equal(only, dx)
    for dtype in (torch.bfloat16, torch.float32):
        old = (torch.randn(V, D, device=dev) * 0.01).to(dtype)
        for ld, at in ((D, 0), (D + 3, 1), ((D + 15) // 8 * 8, 8)):
            buf = strided(old, ld, at)
            around = buf._base.clone() if buf._base is not None else None
            none, got = loss.cross_entropy_grad(x, w, y, lse, g, dw=buf, accumulate=True, needs_dx=False)
            assert none is None and got is buf
            total = dw0 + old.double()
            close(got, total, off_dw + total.abs() * HALF_STEP[dtype] * 1.01 + 1e-37, "dw")
            if around is not None:
                buf.copy_(old)
                assert torch.equal(buf._base, around)     # nothing beside it is written
    ws = strided(w, D + 5, 3)
    dx, dw = loss.cross_entropy_grad(strided(x, D + 1, 1), ws, y, lse, g, dw_dtype=torch.float32)
    close(dx, dx0, off_dx + dx0.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-37, "dx")
    close(dw, dw0, off_dw + dw0.abs() * ULP + 1e-37, "dw")


def test_pieces_of_the_vocabulary(dev):
    """More logits' gradients than the buffer holds: dx is summed over pieces."""
    from weight_communication_gb300 import binding, loss
    for T, V, D in ((4096, 40000, 72), (1000, 300000, 40)):
        x, w, y = inputs(dev, T, V, D, seed=3)
        losses, lse = loss.cross_entropy(x, w, y, save=True)
        dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0 / T, dw_dtype=torch.float32)
        torch.cuda.synchronize()
        assert binding.wait_timeouts() == 0
        want, off = reference(x, w, y, 1.0 / T)
        close(losses, want[0], off[0] + want[0].abs() * 2 * ULP, "losses")
        close(dx, want[2], off[2] + want[2].abs() * HALF_STEP[dx.dtype] * 1.01 + 1e-37, "dx")
        close(dw, want[3], off[3] + want[3].abs() * ULP + 1e-37, "dw")


def test_many_tokens(dev):
    """More than one launch of the forward pass has."""
    from weight_communication_gb300 import loss
    for V, D in ((300, 64), (130, 57)):
        x, w, y = inputs(dev, 140001, V, D, seed=4)
        losses, lse = loss.cross_entropy(x, w, y, save=True)
        want, off = reference(x[:1], w, y[:1], 0.0)
        xd, wd = x.double(), w.double()
        s = xd @ wd.t()
        want = torch.logsumexp(s, 1)
        tol = (D + 16) * 2 * ULP * (xd.abs() @ wd.abs().t()).amax(1) + (want.abs() + s.abs().amax(1) + 128) * 4 * ULP
        close(lse, want, tol, "lse")
        live = (y >= 0) & (y < V)
        sy = s.gather(1, torch.where(live, y, 0)[:, None])[:, 0]
        close(losses, torch.where(live, want - sy, 0.0), 2 * tol, "losses")


def test_offsets_beyond_32_bits(dev):
    """A weight of 2^31 values and more; all rows are 0 but for a few."""
    from weight_communication_gb300 import loss
    V, D = 1100000, 2048
    w = torch.zeros(V, D, device=dev, dtype=torch.bfloat16)
    rows = torch.tensor([0, 5, 1048575, 1048576, 1048577, V - 2, V - 1], device=dev)
    w[rows] = torch.randn(7, D, device=dev).bfloat16()
    for T in (3, 40):
        x = (torch.randn(T, D, device=dev) * 0.05).bfloat16()
        y = rows[torch.arange(T, device=dev) % 7]
        losses, lse = loss.cross_entropy(x, w, y, save=True)
        s = x.double() @ w[rows].double().t()
        want = torch.log(torch.exp(s).sum(1) + (V - 7))
        tol = (D + 16) * 2 * ULP * (x.double().abs() @ w[rows].double().abs().t()).amax(1) + 200 * 4 * ULP
        close(lse, want, tol, "lse")
        close(losses, want - s.gather(1, (torch.arange(T, device=dev) % 7)[:, None])[:, 0], 2 * tol, "losses")
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0)
    d = torch.exp(s - want[:, None])
    d.scatter_add_(1, (torch.arange(T, device=dev) % 7)[:, None], torch.full((T, 1), -1.0, device=dev, dtype=torch.float64))
    off_d = d.abs() * HALF_STEP[torch.bfloat16] * 1.01 + 1e-4 * torch.exp(s - want[:, None])
    close(dx, d @ w[rows].double(), off_d @ w[rows].double().abs() + (d @ w[rows].double()).abs() * 2 ** -8 * 1.01 + 1e-6, "dx")
    want_w = d.t() @ x.double()
    close(dw[rows], want_w, off_d.t() @ x.double().abs() + want_w.abs() * 2 ** -8 * 1.01 + 1e-6, "dw")
    # all other rows have the same gradient: the mean token by 1 / sum
    other = (x.double() / torch.exp(want)[:, None]).sum(0)
    off = (x.double().abs() / torch.exp(want)[:, None]).sum(0) * (2 ** -8 * 2.02 + 1e-4)
    for r in (1, 700001, 1048574, V - 3):
        close(dw[r], other, off + 1e-12, f"row {r}")


def test_padding_holds_anything(dev):
    """A padded token has no loss and no gradient, whatever its row of x holds."""
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, 300, 700, 96, seed=5)
    pad = (y < 0) | (y >= 700)
    want = [loss.cross_entropy(x, w, y)] + list(loss.cross_entropy_grad(x, w, y, loss.cross_entropy(x, w, y, save=True)[1], 0.1))
    x = x.clone()
    x[pad] = torch.tensor([float("nan"), float("inf"), -float("inf")], device=dev).repeat(32).bfloat16()
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 0.1)
    for a, b in zip((losses, dx, dw), want):
        assert torch.equal(a, b)
    assert bool((dx[pad] == 0).all())
    # nothing but padding
    none = torch.full_like(y, -1)
    losses, lse = loss.cross_entropy(x, w, none, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, none, lse, 0.1)
    assert bool((losses == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())


def test_extreme_logits(dev):
    from weight_communication_gb300 import loss
    T, V, D = 260, 1000, 64
    x, w, y = inputs(dev, T, V, D, padding=False, seed=6)
    for scale in (200.0, 1e4, 1e-6):
        xs = (x.float() * scale).bfloat16()
        losses, lse = loss.cross_entropy(xs, w, y, save=True)
        dx, dw = loss.cross_entropy_grad(xs, w, y, lse, 1.0)
        assert bool(losses.isfinite().all()) and bool((losses >= 0).all())
        if scale != 1e4:   # (there the exponentials' own error bound is past 1)
            check(xs, w, y, 1.0, losses, lse, dx, dw)
    # a target far above all others: the loss is their sum over its exponential
    sure = torch.zeros(V, D, device=dev, dtype=torch.bfloat16)
    sure[7, 0] = 16.0
    xs = torch.zeros(4, D, device=dev, dtype=torch.bfloat16)
    xs[:, 0] = torch.tensor([1.0, 1.5, 2.0, 4.0], device=dev)
    for rows in (xs, xs.repeat(3, 1)):
        want = torch.log1p((V - 1) * torch.exp(-16.0 * rows[:, 0].double()))
        got = loss.cross_entropy(rows, sure, torch.full((len(rows),), 7, device=dev))
        # exponentials of up to 64: their arguments' roundings
        close(got, want, want * 1e-5, "losses")
    # an impossible target: its loss is infinite, its gradient that of probability 0
    never = torch.zeros(50, 8, device=dev, dtype=torch.bfloat16)
    never[9, 0] = -float("inf")
    for T2 in (3, 20):
        one = torch.ones(T2, 8, device=dev, dtype=torch.bfloat16)
        y2 = torch.full((T2,), 9, device=dev)
        y2[0] = 3
        got, lse = loss.cross_entropy(one, never, y2, save=True)
        assert bool(got[1:].isinf().all()) and float(got[0]) == pytest.approx(float(torch.tensor(49.0).log()), rel=1e-6)
        close(lse, torch.full((T2,), 49.0, device=dev).log(), torch.full((T2,), 1e-5, device=dev), "lse")
        _, dw = loss.cross_entropy_grad(one, never, y2, lse, 1.0, dw_dtype=torch.float32, needs_dx=False)
        # 1 / 49 in bf16 for each token, -1 for the targets
        want = torch.full((50, 8), T2 / 49.0, device=dev)
        want[9] = 1.0 - T2
        want[3] -= 1.0
        close(dw, want, want.abs() * 2 ** -8 * 1.01 + 2 ** -8 * T2 / 49 * 1.01, "dw")
    # impossible rows, and rows of x that are not finite
    w2 = w.clone()
    w2[11] = 0.0
    w2[11, 0] = -float("inf")
    x2 = x.clone()
    x2[:, 0] = 1.0
    got = loss.cross_entropy(x2, w2, torch.where(y == 11, 12, y))
    keep = torch.arange(V, device=dev) != 11
    s = x2.double() @ w[keep].double().t()
    at = torch.where(y == 11, 12, y)
    sy = (x2.double() * w2[at].double()).sum(1)
    close(got, torch.logsumexp(s, 1) - sy, torch.full((T,), 1e-3, device=dev), "losses")
    x2[3, 5] = float("nan")
    x2[4, 6] = float("inf")
    got = loss.cross_entropy(x2, w, y)
    assert bool(got[3].isnan()) and int(got.isnan().sum()) <= 2 and bool(got[5:].isfinite().all())


def test_gradient_against_differences(dev):
    from weight_communication_gb300 import loss
    T, V, D = 64, 300, 128
    x, w, y = inputs(dev, T, V, D, seed=7)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    g = torch.rand(T, device=dev)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, g, dw_dtype=torch.float32)
    value = lambda a, b: float((loss.cross_entropy(a, b, y).double() * g.double()).sum())  # noqa: E731
    for arg, d in ((x, dx), (w, dw)):
        step = 0.02 * torch.randn(arg.shape, device=dev) * arg.float().abs().mean()
        plus, minus = (arg.float() + step).bfloat16(), (arg.float() - step).bfloat16()
        slope = value(plus, w) - value(minus, w) if arg is x else value(x, plus) - value(x, minus)
        moved = plus.double() - minus.double()
        # the ends' middle is off arg by a rounding (2^-8 of it); the gradient's terms by 2^-8
        # each, at random; the loss is curved over 2 % of the values
        assert slope == pytest.approx(float((d.double() * moved).sum()),
                                      abs=0.05 * float(d.double().norm() * moved.norm()) * 0.3)


def test_shapes_streams_and_graphs(dev):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, 240, 3000, 264, seed=8)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 0.01)
    a, b = loss.cross_entropy(x.view(4, 60, 264), w, y.view(4, 60), save=True)
    assert a.shape == b.shape == (4, 60) and torch.equal(a.view(-1), losses)
    c, _ = loss.cross_entropy_grad(x.view(4, 60, 264), w, y.view(4, 60), b, 0.01)
    assert c.shape == (4, 60, 264) and torch.equal(c.view(240, 264), dx)
    e = torch.empty(0, 264, device=dev, dtype=torch.bfloat16)
    n = torch.empty(0, device=dev, dtype=torch.int64)
    a, b = loss.cross_entropy(e, w, n, save=True)
    c, d = loss.cross_entropy_grad(e, w, n, b, 0.01)
    assert a.shape == (0,) and c.shape == (0, 264) and bool((d == 0).all())
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(3):
        a, b = loss.cross_entropy(x, w, y, save=True, stream=s)
        c, d = loss.cross_entropy_grad(x, w, y, b, 0.01, stream=s)
        junk = torch.full((3000, 264), 7.0, device=dev)  # on the default stream
        del junk
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in ((a, losses), (b, lse), (c, dx), (d, dw)))
    # two graphs, replayed in turn and side by side
    graphs, outs, xs = [], [], []
    for k in range(2):
        xk = torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a, b = loss.cross_entropy(xk, w, y, save=True)
            c, d = loss.cross_entropy_grad(xk, w, y, b, 0.01)
        graphs.append(graph)
        outs.append((a, b, c, d))
        xs.append(xk)
    xs[0].copy_(x)
    xs[1].copy_(x.roll(1, 0))
    one = loss.cross_entropy(xs[1], w, y, save=True)
    other = (*one, *loss.cross_entropy_grad(xs[1], w, y, one[1], 0.01))
    other_stream = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(other_stream):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs[0], (losses, lse, dx, dw)))
        assert all(torch.equal(p, q) for p, q in zip(outs[1], other))


def test_one_gradient_for_all_is_not_rounded(dev):
    """dlosses as one number multiplies the products: scaling by it commutes."""
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, 200, 500, 64, seed=9)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0, dw_dtype=torch.float32)
    dx2, dw2 = loss.cross_entropy_grad(x, w, y, lse, 1.0 / 3, dw_dtype=torch.float32)
    third = torch.tensor(1.0 / 3, dtype=torch.float32, device=dev)
    assert torch.equal(dw2, dw * third)
    close(dx2, dx.double() * third.double(), dx.double().abs() * 2 ** -8 * 1.5 + 1e-37, "dx")


def test_refusals(dev):
    from weight_communication_gb300 import loss
    x, w, y = inputs(dev, 20, 100, 64, seed=10)
    _, lse = loss.cross_entropy(x, w, y, save=True)
    for bad, kind, match in ((dict(x=x.float()), TypeError, "x must be"), (dict(w=w.float()), TypeError, "weight must be"),
                             (dict(w=w[:, :63]), ValueError, "weight has shape"), (dict(w=w.cpu()), ValueError, "weight is on"),
                             (dict(w=w[0]), ValueError, "weight has shape"), (dict(y=y.float()), TypeError, "targets must be"),
                             (dict(y=y[:19]), ValueError, "targets has shape"), (dict(y=y.cpu()), ValueError, "targets is on"),
                             (dict(y=torch.stack([y, y], 1)[:, 0]), ValueError, "contiguous"),
                             (dict(w=torch.zeros(64, 100, device=dev, dtype=torch.bfloat16).t()), ValueError, "consecutive")):
        a = dict(x=x, w=w, y=y)
        a.update(bad)
        with pytest.raises(kind, match=match):
            loss.cross_entropy(a["x"], a["w"], a["y"])
        with pytest.raises(kind, match=match):
            loss.cross_entropy_grad(a["x"], a["w"], a["y"], lse, 1.0)
    for args, kw, kind, match in (((lse[:19], 1.0), {}, ValueError, "lse has shape"), ((lse.double(), 1.0), {}, TypeError, "lse must be"),
                                  ((lse, lse[:3]), {}, ValueError, "dlosses has shape"), ((lse, "a"), {}, TypeError, "number"),
                                  ((lse, 1.0), dict(accumulate=True), ValueError, "accumulate needs"),
                                  ((lse, 1.0), dict(dw=w[:50].clone()), ValueError, "dw has shape"),
                                  ((lse, 1.0), dict(dw=w.half()), TypeError, "dw must be"),
                                  ((lse, 1.0), dict(dw=w.clone(), dw_dtype=torch.float32), TypeError, "dw must be"),
                                  ((lse, 1.0), dict(dw_dtype=torch.float16), TypeError, "dw_dtype"),
                                  ((lse, 1.0), dict(needs_dx=False, needs_dw=False), ValueError, "neither"),
                                  ((lse, 1.0), dict(needs_dw=False, dw=w.clone()), ValueError, "not asked for")):
        with pytest.raises(kind, match=match):
            loss.cross_entropy_grad(x, w, y, *args, **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,V,D", [(70, 700, 1100), (300, 2000, 2048), (257, 511, 2500), (5, 130, 9001), (600, 900, 4500),
                                   (20, 3000, 8200), (130, 20000, 1032)])
def test_long_rows(dev, T, V, D):
    """Rows whose products are summed in several chunks."""
    from weight_communication_gb300 import binding, loss
    x, w, y = inputs(dev, T, V, D, seed=11)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    dx, dw = loss.cross_entropy_grad(x, w, y, lse, 1.0 / T)
    torch.cuda.synchronize()
    assert binding.wait_timeouts() == 0
    check(x, w, y, 1.0 / T, losses, lse, dx, dw)
    assert torch.equal(loss.cross_entropy(x, w, y), losses)


@pytest.mark.parametrize("D", [1024, 4096, 16384, 50000])
def test_what_sums_lose_does_not_grow_with_the_row(dev, D):
    """Products of one sign, whose sums only grow: what each step cuts off adds up."""
    from weight_communication_gb300 import loss
    g = torch.Generator(device=dev)
    g.manual_seed(D)
    x = torch.rand(8, D, generator=g, device=dev).add_(0.5).bfloat16()
    w = (torch.rand(300, D, generator=g, device=dev).add_(0.5) * (6 / D)).bfloat16()
    y = torch.arange(8, device=dev)
    losses, lse = loss.cross_entropy(x, w, y, save=True)
    s = x.double() @ w.double().t()
    want = torch.logsumexp(s, 1)
    # 64 steps of 16 values to a chunk, each of which may lose an ulp of what is summed so
    # far; a rounding for each chunk that is added; and those of the exponentials and
    # logarithms, at arguments of up to 64
    off = s.amax(1) * (64 * 2 ** -23 + -(-D // 1024) * 2 ** -24) + 64 * 4 * 2 ** -24
    close(lse, want, off, "lse")
    close(losses, want - s[torch.arange(8), y], off + s.amax(1) * D ** 0.5 * 2 ** -24, "losses")
