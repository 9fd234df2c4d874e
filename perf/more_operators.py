"""Measured cases of the operators between a training step's layers, and of its loss.

  * loss / loss_train: softmax cross entropy of a linear output layer over the
    vocabulary, in pieces of the vocabulary and without keeping the logits --
    the tokens' losses and log-sums alone, or with the gradients of activations and weight;
  * act / act_train: a layer's activation (gated or not) -- alone, or kept in
    8 bits by the forward pass with the backward pass that reads it;
  * norm / norm_train: root-mean-square norm of a residual stream, likewise;
  * restore: a matrix kept in 8 bits back to its values.

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, by the calls a user makes of weight_communication_gb300.  `exact` states
them again in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # values per scale, along a row
TOP = 448.0          # largest e4m3 value
TINY = 2.0 ** -126   # smallest normal binary32
EPS = 1e-6           # added to the mean square
EXACT_FLOPS = 4e12   # of a 64-bit product; more take too long


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # scoring one token against the 32000 x 2048 output layer: latency, one reading of the weight
        dict(name="loss_1_token", op="loss", T=1, V=32000, D=2048, wide=True),
        # evaluation of a short batch, no size a multiple of a tile, rows that start anywhere
        dict(name="loss_odd", op="loss", T=333, V=12501, D=1001, wide=False),
        # a micro-batch's loss and gradients, d = 2048 and 32000 rows: the largest
        dict(name="loss_train_8k", op="loss_train", T=8192, V=32000, D=2048, wide=True),
        # training at odd, ragged sizes, one target in eight padding
        dict(name="loss_train_odd", op="loss_train", T=777, V=10007, D=1003, wide=False),
        # one token through the d = 2048 layer's gated activation: latency
        dict(name="act_1_token", op="act", rows=1, cols=5504, kind="silu", gated=True, dtype="bf16"),
        # a micro-batch through the d = 4096 layer's gated activation, both ways
        dict(name="act_train_8k", op="act_train", rows=8192, cols=11008, kind="silu", gated=True,
             dtype="bf16"),
        # odd sizes, fp32, not gated
        dict(name="act_train_odd", op="act_train", rows=333, cols=1003, kind="gelu", gated=False,
             dtype="f32"),
        # one token's norm with its residual sum, d = 2048: latency
        dict(name="norm_1_token", op="norm", rows=1, cols=2048, add=True, dtype="bf16"),
        # a micro-batch's norm with its residual sum, d = 4096, both ways
        dict(name="norm_train_8k", op="norm_train", rows=8192, cols=4096, add=True, dtype="bf16"),
        # odd sizes, fp32, without a residual
        dict(name="norm_train_odd", op="norm_train", rows=777, cols=1501, add=False, dtype="f32"),
        # the d = 4096 layer's hidden activation back from 8 bits
        dict(name="restore_8k", op="restore", rows=8192, cols=11008, dtype="bf16"),
        # the same at odd sizes, to fp32
        dict(name="restore_odd", op="restore", rows=333, cols=1003, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss_train", "loss_train", "act", "act_train", "norm", "norm_train",
                     "restore"])
    if op in ("loss", "loss_train"):
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), V=_log(rng, 500, 64000), D=_log(rng, 64, 4096),
                     wide=rng.random() < 0.5)
            if c["T"] * c["V"] * c["D"] <= 8192 * 32000 * 2048:
                return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 11008), dtype=dtype)
    if op in ("act", "act_train"):
        c.update(kind=rng.choice(["silu", "gelu", "relu"]), gated=rng.random() < 0.7)
    elif op in ("norm", "norm_train"):
        c.update(cols=_log(rng, 64, 8192), add=rng.random() < 0.6)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _normal(shape, sigma, g, dtype=torch.bfloat16, outliers=0.0):
    """N(0, sigma^2), a fraction of the values 20 times as large."""
    x = torch.randn(shape, generator=g, device=DEV) * sigma
    if outliers:
        x = torch.where(torch.rand(shape, generator=g, device=DEV) < outliers, x * 20.0, x)
    return x.to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("loss", "loss_train"):
        T, V, D = case["T"], case["V"], case["D"]
        w = _normal((V, D), 0.02, g)
        # targets with Zipf's law; one in eight of a training batch is padding
        u = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
        targets = ((u * math.log(V + 1)).exp().long() - 1).clamp(0, V - 1)
        # the model knows some tokens: a push of 0 to 8 towards the target's logit
        push = torch.rand(T, 1, generator=g, device=DEV) * (8.0 / (D * 4e-4))
        x = (torch.randn(T, D, generator=g, device=DEV) + push * w[targets].float()).to(torch.bfloat16)
        if op == "loss_train":
            pad = torch.rand(T, generator=g, device=DEV) < 0.125
            targets = torch.where(pad, torch.full_like(targets, -100), targets)
        return dict(case=case, x=x, w=w, targets=targets if case["wide"] else targets.int(),
                    dloss=1.0 / max(1.0, round(0.875 * T)))
    rows, cols = case["rows"], case["cols"]
    t = _type(case["dtype"])
    if op in ("act", "act_train"):
        st = dict(case=case, gate=_normal((rows, cols), 1.5, g, t, 1e-3),
                  up=_normal((rows, cols), 1.0, g, t, 1e-3) if case["gated"] else None)
        if op == "act_train":
            st["dh"] = _normal((rows, cols), 1e-3, g, t, 1e-4)
        return st
    if op in ("norm", "norm_train"):
        st = dict(case=case, x=_normal((rows, cols), 2.0, g, t, 1e-3),
                  add=_normal((rows, cols), 0.5, g, t) if case["add"] else None,
                  weight=(1.0 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(t))
        if op == "norm_train":
            st["dy"] = _normal((rows, cols), 1e-3, g, t, 1e-4)
            # what reaches the sum past the norm
            st["dtotal"] = _normal((rows, cols), 1e-3, g, t) if case["add"] else None
        return st
    x = _normal((rows, cols), 1.0, g, torch.bfloat16, 1e-3)
    codes, scales = _coded(x.float())
    ld = -(-cols // 16) * 16
    kept = torch.zeros(rows, ld, dtype=torch.uint8, device=DEV)     # rows start on 16 bytes
    kept[:, :cols] = codes.view(torch.uint8)
    return dict(case=case, codes=kept.view(torch.float8_e4m3fn), scales=scales.t().contiguous())


# ---------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _coded(x):
    """x [R, C] fp32 in e4m3 with a scale per 128 of a row: codes [R, C] and
    scales [R, C / 128].  The values next to a border between two codes fall
    as one binary32 division and one binary32 product say."""
    r, c = x.shape
    cb = -(-c // BLOCK)
    p = x.new_zeros(r, cb * BLOCK)
    p[:, :c] = x
    p = p.view(r, cb, BLOCK)
    m = p.abs().amax(dim=2)
    live = m >= TOP * TINY
    safe, top = torch.where(live, m, torch.ones_like(m)), torch.full_like(m, TOP)
    # tensor by tensor: a division by a Python number is a product with its
    # rounded reciprocal, which moves codes
    s = torch.where(live, m / top, torch.zeros_like(m))
    inv = torch.where(live, top / safe, torch.zeros_like(m))
    q = (p * inv[:, :, None]).to(torch.float8_e4m3fn).view(r, cb * BLOCK)
    return q[:, :c], s


def _values(codes, scales):
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _kept(x):
    """What fp32 x stands for after a stay in 8 bits."""
    return _values(*_coded(x))


def _act(kind, a):
    """act(a) and its derivative."""
    if kind == "relu":
        on = (a > 0).to(a.dtype)
        return a * on, on
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 0.134145 * a * a)


def _plain_loss(st):
    V = st["case"]["V"]
    x, w = st["x"].float(), st["w"].float()
    s = x @ w.t()
    top = s.amax(dim=1, keepdim=True)
    e = torch.exp(s - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    y = st["targets"].long()
    live = (y >= 0) & (y < V)
    at = torch.where(live, y, torch.zeros_like(y))[:, None]
    losses = torch.where(live, lse - s.gather(1, at)[:, 0], torch.zeros_like(lse))
    if st["case"]["op"] == "loss":
        return {"losses": losses, "lse": lse}
    p = e.div_(total)
    p.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    p *= torch.where(live, st["dloss"], 0.0)[:, None]
    return {"losses": losses, "dx": (p @ w).to(torch.bfloat16), "dw": (p.t() @ x).to(torch.bfloat16)}


def _plain_act(st):
    c = st["case"]
    t = _type(c["dtype"])
    gate = st["gate"].float()
    up = st["up"].float() if c["gated"] else None
    h = _act(c["kind"], gate)[0]
    h = (h * up if c["gated"] else h).to(t)
    if c["op"] == "act":
        return h
    a, da = _act(c["kind"], _kept(gate))
    dh = st["dh"].float()
    if not c["gated"]:
        return {"h": h, "dgate": (dh * da).to(t)}
    return {"h": h, "dgate": (dh * _kept(up) * da).to(t), "dup": (dh * a).to(t)}


def _plain_norm(st):
    c = st["case"]
    t = _type(c["dtype"])
    total = (st["x"].float() + st["add"].float()).to(t) if c["add"] else st["x"]
    x, w = total.float(), st["weight"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    out = {"y": (x * rstd * w).to(t)}
    if c["add"]:
        out["total"] = total
    if c["op"] == "norm":
        return out
    n = _kept(x) * rstd
    dy = st["dy"].float()
    wd = dy * w
    dx = rstd * (wd - n * (wd * n).mean(dim=1, keepdim=True))
    if c["add"]:
        dx = dx + st["dtotal"].float()
    out["dx"], out["dweight"] = dx.to(t), (dy * n).sum(dim=0)
    return out


def _plain_restore(st):
    c = st["case"]
    return _values(st["codes"][:, :c["cols"]], st["scales"].t()).to(_type(c["dtype"]))


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_loss(st):
    from weight_communication_gb300 import loss
    losses, lse = loss.cross_entropy(st["x"], st["w"], st["targets"], save=True)
    if st["case"]["op"] == "loss":
        return {"losses": losses, "lse": lse}
    dx, dw = loss.cross_entropy_grad(st["x"], st["w"], st["targets"], lse, st["dloss"])
    return {"losses": losses, "dx": dx, "dw": dw}


def _own_act(st):
    from weight_communication_gb300 import activation
    c = st["case"]
    if c["op"] == "act":
        return activation.forward(st["gate"], st["up"], kind=c["kind"])
    h, kept = activation.forward(st["gate"], st["up"], kind=c["kind"], save=True)
    dgate, dup = activation.backward(st["dh"], kept)
    return {"h": h, "dgate": dgate, "dup": dup} if c["gated"] else {"h": h, "dgate": dgate}


def _own_norm(st):
    from weight_communication_gb300 import norm
    c = st["case"]
    if c["op"] == "norm":
        y, total = norm.rms(st["x"], st["weight"], eps=EPS, add=st["add"])
        return {"y": y, "total": total} if c["add"] else {"y": y}
    y, total, kept = norm.rms(st["x"], st["weight"], eps=EPS, add=st["add"], save=True)
    dx, dweight = norm.rms_grad(st["dy"], st["weight"], kept, add=st["dtotal"])
    out = {"y": y, "total": total} if c["add"] else {"y": y}
    out["dx"], out["dweight"] = dx, dweight
    return out


def _own_restore(st):
    from weight_communication_gb300 import fp8
    c = st["case"]
    q = fp8.Fp8Tensor(st["codes"], st["scales"], c["rows"], c["cols"])
    return fp8.dequantize(q, _type(c["dtype"]))


PLAIN = {"loss": _plain_loss, "act": _plain_act, "norm": _plain_norm, "restore": _plain_restore}
OWN = {"loss": _own_loss, "act": _own_act, "norm": _own_norm, "restore": _own_restore}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"].removesuffix("_train")](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("loss", "loss_train"):
        T, V, D = case["T"], case["V"], case["D"]
        read = 2 * (T * D + V * D) + (8 if case["wide"] else 4) * T + 4 * T
        if op == "loss":
            return {"bytes": read + 4 * T, "flops": 2 * T * V * D}
        # the logits once (that they are not kept, and so multiplied twice, is
        # the operator's own price), and the two gradients
        return {"bytes": read + 2 * (T * D + V * D), "flops": 6 * T * V * D}
    n = case["rows"] * case["cols"]
    e = {"bf16": 2, "f32": 4}[case["dtype"]]
    kept = n + 4 * case["rows"] * (-(-case["cols"] // BLOCK))
    if op == "restore":
        return {"bytes": kept + n * e, "flops": n}
    if op in ("act", "act_train"):
        parts = 2 if case["gated"] else 1
        if op == "act":
            return {"bytes": (parts + 1) * n * e, "flops": 8 * n}
        # what is kept is written by one pass and read by the other
        return {"bytes": (2 * parts + 2) * n * e + 2 * parts * kept, "flops": 24 * n}
    through = (4 if case["add"] else 2) * n * e
    if op == "norm":
        return {"bytes": through + case["cols"] * e, "flops": 5 * n}
    back = (3 if case["add"] else 2) * n * e
    return {"bytes": through + back + 2 * kept + case["cols"] * (2 * e + 4) + 8 * case["rows"],
            "flops": 14 * n}


def _exact_kept(x):
    """The 64-bit values that x [R, C] stands for in 8 bits, by the spacing of
    each value's binade.  Which code a value gets is defined by one binary32
    division and one binary32 product; all else is in 64 bits."""
    r, c = x.shape
    wide = -(-c // BLOCK) * BLOCK
    p = torch.nn.functional.pad(x.float(), (0, wide - c)).view(r, wide // BLOCK, BLOCK)
    m = p.abs().amax(2)
    dead = m < TOP * TINY
    inv = (torch.full_like(m, TOP) / m.masked_fill(dead, 1.0)).masked_fill(dead, 0.0)
    scale = (m / torch.full_like(m, TOP)).masked_fill(dead, 0.0)
    v = (p * inv.unsqueeze(2)).double()
    _, exponent = torch.frexp(v)
    step = torch.exp2((exponent - 1).clamp(min=-6).double() - 3)
    codes = torch.round(v / step).mul_(step).clamp_(-TOP, TOP)
    return (codes * scale.double().unsqueeze(2)).view(r, wide)[:, :c]


def _exact_loss(st, case):
    T, V, D = case["T"], case["V"], case["D"]
    if T * V * D * (2 if case["op"] == "loss" else 6) > EXACT_FLOPS:
        return None
    x, w = st["x"].double(), st["w"].double()
    s = torch.einsum("td,vd->tv", x, w)
    lse = torch.logsumexp(s, 1)
    here = ((st["targets"] >= 0) & (st["targets"] < V)).nonzero()[:, 0]
    at = st["targets"].long()[here]
    losses = torch.zeros(T, dtype=torch.float64, device=DEV)
    losses[here] = lse[here] - s[here, at]
    if case["op"] == "loss":
        return {"losses": losses, "lse": lse}
    d = torch.zeros_like(s)
    d[here] = torch.softmax(s[here], 1)
    d[here, at] = torch.expm1(s[here, at] - lse[here])
    d *= st["dloss"]
    return {"losses": losses, "dx": torch.einsum("tv,vd->td", d, w), "dw": torch.einsum("tv,td->vd", d, x)}


def _exact_act(kind, a):
    """act(a) and its derivative, by autograd of the definition in 64 bits."""
    a = a.detach().requires_grad_()
    with torch.enable_grad():
        if kind == "relu":
            f = torch.relu(a)
        elif kind == "silu":
            f = a * torch.sigmoid(a)
        else:
            f = a * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3))
        d, = torch.autograd.grad(f.sum(), a)
    return f.detach(), d


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("loss", "loss_train"):
        return _exact_loss(st, case)
    if op == "restore":
        cols = case["cols"]
        s = st["scales"].double()[torch.arange(cols, device=DEV) // BLOCK]
        return st["codes"][:, :cols].float().double() * s.t()
    if op in ("act", "act_train"):
        f, _ = _exact_act(case["kind"], st["gate"].double())
        h = f * st["up"].double() if case["gated"] else f
        if op == "act":
            return h
        f, d = _exact_act(case["kind"], _exact_kept(st["gate"]))
        dh = st["dh"].double()
        if not case["gated"]:
            return {"h": h, "dgate": dh * d}
        return {"h": h, "dgate": dh * d * _exact_kept(st["up"]), "dup": dh * f}
    total = st["x"]
    if case["add"]:   # defined by the type's own sum
        total = (total.float() + st["add"].float()).to(_type(case["dtype"]))
    x, w = total.double(), st["weight"].double()
    rstd = torch.rsqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / case["cols"] + EPS)
    out = {"y": x * rstd * w}
    if case["add"]:
        out["total"] = total
    if op == "norm":
        return out
    n = _exact_kept(total) * rstd
    dy = st["dy"].double()
    dx = (dy * w - n * (torch.einsum("rc,rc->r", dy * w, n) / case["cols"])[:, None]) * rstd
    out["dx"] = dx + st["dtotal"].double() if case["add"] else dx
    out["dweight"] = torch.einsum("rc,rc->c", dy, n)
    return out
