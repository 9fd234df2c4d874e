"""64-bit statements of the operators between the layers, for their tests."""
import math

import torch

TOP, TINY = 448.0, 2.0 ** -126
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ULP = 2.0 ** -24


def kept(x):
    """The 64-bit values that x [R, C] stands for in e4m3 with a scale per 128 of a
    row: codes by one binary32 division and one binary32 product."""
    r, c = x.shape
    wide = -(-max(c, 1) // 128) * 128
    p = torch.nn.functional.pad(x.float(), (0, wide - c)).view(r, wide // 128, 128)
    m = p.abs().amax(2) if r else p.new_zeros(0, wide // 128)
    bad = ~torch.isfinite(m) | p.isnan().any(2)
    dead = (m < TOP * TINY) | bad
    inv = (torch.full_like(m, TOP) / m.masked_fill(dead, 1.0)).masked_fill(dead, 0.0)
    scale = (m / torch.full_like(m, TOP)).masked_fill(dead, 0.0).double().masked_fill(bad, math.nan)
    v = (p * inv.unsqueeze(2)).nan_to_num(0.0).to(torch.float8_e4m3fn).double()
    return (v * scale.unsqueeze(2)).view(r, wide)[:, :c]


def act(kind, a):
    """act(a), its derivative, and bounds of what fp32 may be off by in each."""
    a = a.double()
    if kind == "relu":
        d = (a > 0).double().masked_fill(a.isnan(), math.nan)
        return torch.where(a < 0, torch.zeros_like(a), a), d, torch.zeros_like(a), torch.zeros_like(a)
    k = 2.0 * math.sqrt(2.0 / math.pi)
    z, dz = (a, torch.ones_like(a)) if kind == "silu" else (k * (a + 0.044715 * a ** 3), k * (1 + 0.134145 * a * a))
    s = torch.sigmoid(z)
    d = s + torch.where(z.abs() > 700, torch.zeros_like(a), a * s * torch.sigmoid(-z) * dz)
    # exponentials: 2 ulp, and z's own roundings (three of them, and one of z
    # log2 e) count with z itself; then a sum, a reciprocal and two products
    rel = (16 + 6 * z.abs().clamp(max=200)) * ULP
    # a sigmoid below the smallest normal number, 2^-126, may come as 0: that
    # times |a| is lost of the first, and times 1 + |a z'| of the second
    lost = rel * s + TINY
    # s (1 + a (1 - s) z'): each factor as above
    return a * s, d, a.abs() * lost, (lost + 4 * ULP * s) * (1 + 2 * (a * dz).abs().nan_to_num(0.0).clamp(max=1e30))


def close(got, want, tol, what=""):
    """|got - want| <= tol everywhere, and NaN in the same places."""
    got, want, tol = got.double(), want.double(), tol.double()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    off = torch.where(got == want, torch.zeros_like(got), (got - want).abs()).nan_to_num(0.0, posinf=math.inf)
    bad = off > tol.nan_to_num(math.inf)
    if bool(bad.any()):
        i = int((off / tol.clamp(min=1e-300)).masked_fill(~bad, 0.0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} values off, the worst {got.reshape(-1)[i]} "
                             f"for {want.reshape(-1)[i]} (allowed {tol.reshape(-1)[i]}) at {i}")


def strided(x, ld, offset=0):
    """x [R, C] with rows ld apart, starting `offset` values into its memory."""
    r, c = x.shape
    flat = torch.full((offset + r * ld + ld,), 3.0, dtype=x.dtype, device=x.device)
    v = flat[offset:offset + r * ld].view(r, ld)[:, :c]
    v.copy_(x)
    return v
