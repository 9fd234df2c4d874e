"""Measured cases of the training-step operators around the gradient exchange.

Three operators of one data-parallel training step:

  * linear / train: the matrix product in 8-bit floating point (e4m3) with one
    fp32 scale per block of 128 -- forward with kept 8-bit weights, and the
    whole training form (weights, activations and gradients quantized within
    the pass, y, dx and dw returned);
  * embed / embed_grad: the embedding lookup with scaling, and its gradient
    summed over the tokens of each row;
  * clip: the global gradient norm over many tensors and the clipping.

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, by the calls a user makes of weight_communication_gb300.  `exact` states
them again in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # values per scale, along the summed axis
TOP = 448.0          # largest e4m3 value
TINY = 2.0 ** -126   # smallest normal binary32
EPS = 1e-6           # added to the norm before the division


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through the up projection of the d=2048 layer: latency
        dict(name="linear_1_token", op="linear", M=1, N=5504, K=2048),
        # a short odd batch, no size a multiple of a tile or of 128
        dict(name="linear_odd", op="linear", M=333, N=1003, K=1501),
        # long batch through the up projection of the d=4096 layer: the largest
        dict(name="linear_8k_tokens", op="linear", M=8192, N=11008, K=4096),
        # one training step of the d=2048 layer's up projection
        dict(name="train_4k_tokens", op="train", M=4096, N=5504, K=2048),
        # training at odd, ragged sizes
        dict(name="train_odd", op="train", M=777, N=1111, K=555),
        # lookup of a micro-batch in the 32000 x 2048 table
        dict(name="embed_8k_tokens", op="embed", n=8192, V=32000, D=2048, dtype="bf16", wide=True,
             first=0, scale=1.0),
        # a few tokens from an fp32 shard of the vocabulary, odd row length
        dict(name="embed_odd", op="embed", n=37, V=12501, D=1001, dtype="f32", wide=False,
             first=12501, scale=31.5),
        # gradient of a micro-batch, dense bf16 gradient of the whole table
        dict(name="embed_grad_16k", op="embed_grad", n=16384, V=32000, D=2048, dtype="bf16",
             gdtype="bf16", wide=True, first=0, scale=1.0, accumulate=False),
        # fp32 gradient accumulated over micro-batches, odd sizes
        dict(name="embed_grad_odd", op="embed_grad", n=3001, V=50021, D=1002, dtype="bf16",
             gdtype="f32", wide=False, first=0, scale=4.0, accumulate=True),
        # the four fp32 shards of the smallest reduce (1 M elements): latency
        dict(name="clip_1m_f32", op="clip", layers=0, d=0, ffn=0, vocab=0, n=1048576, parts=4,
             src="f32", dst="f32", inplace=False, clipped=True),
        # one d=2048 layer, bf16 gradients clipped into the optimizer's fp32 ones
        dict(name="clip_layer", op="clip", layers=1, d=2048, ffn=5504, vocab=0, n=0, parts=0,
             src="bf16", dst="f32", inplace=False, clipped=True),
        # the 16-layer model with its embedding (875 M), in place, norm within the bound
        dict(name="clip_model", op="clip", layers=16, d=2048, ffn=5504, vocab=32000, n=0, parts=0,
             src="bf16", dst="bf16", inplace=True, clipped=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "train", "embed", "embed_grad", "clip"])
    if op == "linear":
        while True:
            c = dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 200, 11008), K=_log(rng, 200, 11008))
            if c["M"] * c["N"] * c["K"] <= 8192 * 11008 * 4096:
                return c
    if op == "train":
        while True:
            c = dict(op=op, M=_log(rng, 64, 8192), N=_log(rng, 200, 11008), K=_log(rng, 200, 11008))
            if 3 * c["M"] * c["N"] * c["K"] <= 8192 * 11008 * 4096:
                return c
    if op in ("embed", "embed_grad"):
        V = _log(rng, 1000, 64000)
        c = dict(op=op, n=_log(rng, 1, 32768), V=V, D=_log(rng, 64, 4096),
                 dtype=rng.choice(["bf16", "f32"]), wide=rng.random() < 0.5,
                 first=rng.choice([0, 0, V]), scale=rng.choice([1.0, 45.25, 0.5]))
        if op == "embed_grad":
            c.update(gdtype=rng.choice(["bf16", "f32"]), accumulate=rng.random() < 0.4)
        return c
    kind = rng.random()
    src = rng.choice(["bf16", "f32"])
    inplace = rng.random() < 0.4
    c = dict(op="clip", layers=0, d=0, ffn=0, vocab=0, n=0, parts=0, src=src,
             dst=src if inplace else rng.choice(["bf16", "f32"]), inplace=inplace,
             clipped=not inplace)
    if kind < 0.5:
        c.update(n=_log(rng, 1000, 1 << 28), parts=rng.randint(1, 300))
    else:
        c.update(layers=rng.randint(1, 8), d=_log(rng, 256, 2048), ffn=_log(rng, 700, 5504),
                 vocab=_log(rng, 1000, 32000))
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


def _normal(shape, sigma, g, outliers=0.0):
    """N(0, sigma^2), a fraction of the values 20 times as large, in bf16."""
    x = torch.randn(shape, generator=g, device=DEV) * sigma
    if outliers:
        x = torch.where(torch.rand(shape, generator=g, device=DEV) < outliers, x * 20.0, x)
    return x.to(torch.bfloat16)


def _spans(case):
    """Element counts of the tensors of one list, in order."""
    if case["parts"]:
        n, p = case["n"], case["parts"]
        cuts = [n * i // p for i in range(p + 1)]
        return [b - a for a, b in zip(cuts, cuts[1:])]
    d, f = case["d"], case["ffn"]
    layer = [d * d] * 4 + [d * f] * 3 + [d] * 2
    return layer * case["layers"] + ([case["vocab"] * d, d] if case["vocab"] else [])


def _views(flat, counts):
    out, at = [], 0
    for n in counts:
        out.append(flat[at:at + n])
        at += n
    return out


def _ids(case, g):
    """Token ids with Zipf's law (the k-th most frequent has a share of about
    1/k), the table's rows starting at `first`; one in fifty is padding (-1),
    and where the table is a shard some belong to another shard."""
    n, V, first = case["n"], case["V"], case["first"]
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    ids = ((u * math.log(V + 1)).exp().long() - 1).clamp(0, V - 1) + first
    r = torch.rand(n, generator=g, device=DEV)
    if first:
        ids = torch.where(r < 0.3, ids - first, ids)
    ids = torch.where(r > 0.98, -torch.ones_like(ids), ids)
    return ids if case["wide"] else ids.int()


def _fp8_block_weight(w):
    """A weight as it is kept in 8 bits: codes and one scale per 128 x 128."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
    p[:n, :k] = w.float()
    p = p.view(nb, BLOCK, kb, BLOCK)
    m = p.abs().amax(dim=(1, 3))
    s, inv = _scale(m)
    q = (p * inv[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)
    return q[:n, :k], s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _normal((M, K), 1.0, g, 1e-3)
        codes, scales = _fp8_block_weight(_normal((N, K), 0.02, g))
        ld = -(-K // 16) * 16
        kept = torch.zeros(N, ld, dtype=torch.uint8, device=DEV)   # rows start on 16 bytes
        kept[:, :K] = codes.view(torch.uint8)
        return dict(case=case, x=x, codes=kept.view(torch.float8_e4m3fn),
                    scales=scales.t().contiguous())               # [K/128, N/128]
    if op == "train":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(case=case, x=_normal((M, K), 1.0, g, 1e-3), w=_normal((N, K), 0.02, g),
                    dy=_normal((M, N), 1e-3, g, 1e-4))
    if op == "embed":
        t = _normal((case["V"], case["D"]), 0.02, g).to(_type(case["dtype"]))
        return dict(case=case, table=t, ids=_ids(case, g))
    if op == "embed_grad":
        dy = _normal((case["n"], case["D"]), 1e-3, g, 1e-4).to(_type(case["dtype"]))
        st = dict(case=case, dy=dy, ids=_ids(case, g))
        if case["accumulate"]:
            # the gradient of the earlier micro-batches: each pass adds to it
            st["grad"] = _normal((case["V"], case["D"]), 1e-3, g).to(_type(case["gdtype"]))
        return st
    counts = _spans(case)
    flat = _normal((sum(counts),), 1e-3, g, 1e-4).to(_type(case["src"]))
    out = flat if case["inplace"] else torch.empty(flat.numel(), dtype=_type(case["dst"]), device=DEV)
    norm = math.sqrt(flat.numel()) * 1e-3
    st = dict(case=case, flat=flat, grads=_views(flat, counts), out=out,
              outs=_views(out, counts), max_norm=0.25 * norm if case["clipped"] else 8.0 * norm)
    if own:
        # a program names its gradient buffers once, before its first step
        from weight_communication_gb300 import gradnorm
        st["list"] = gradnorm.TensorList(st["grads"])
        st["out_list"] = None if case["inplace"] else gradnorm.TensorList(st["outs"])
    return st


# ---------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _scale(m):
    """scale = m / 448 and 448 / m of blocks with largest magnitude m; blocks
    whose scale would not be a normal number are zero."""
    live = m >= TOP * TINY
    safe, top = torch.where(live, m, torch.ones_like(m)), torch.full_like(m, TOP)
    # tensor by tensor: a division by a Python number is a product with its
    # rounded reciprocal, which moves codes
    return (torch.where(live, m / top, torch.zeros_like(m)),
            torch.where(live, top / safe, torch.zeros_like(m)))


def _rounded(x):
    """What x [R, C] stands for after e4m3 with a scale per 128 of a row."""
    r, c = x.shape
    cb = -(-c // BLOCK)
    p = x.new_zeros(r, cb * BLOCK)
    p[:, :c] = x
    p = p.view(r, cb, BLOCK)
    s, inv = _scale(p.abs().amax(dim=2))
    q = (p * inv[:, :, None]).to(torch.float8_e4m3fn).float() * s[:, :, None]
    return q.view(r, cb * BLOCK)[:, :c]


def _spread(scales, n, k):
    return scales.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _plain_linear(st):
    N, K = st["case"]["N"], st["case"]["K"]
    w = st["codes"][:, :K].float() * _spread(st["scales"].t(), N, K)
    return (_rounded(st["x"].float()) @ w.t()).to(torch.bfloat16)


def _plain_train(st):
    x, dy = st["x"].float(), st["dy"].float()
    codes, s = _fp8_block_weight(st["w"])
    w = codes.float() * _spread(s, *st["w"].shape)
    y = (_rounded(x) @ w.t()).to(torch.bfloat16)
    dx = (_rounded(dy) @ w).to(torch.bfloat16)
    dw = _rounded(dy.t()) @ _rounded(x.t()).t()
    return {"y": y, "dx": dx, "dw": dw}


def _plain_embed(st):
    c = st["case"]
    row = st["ids"].long() - c["first"]
    live = (row >= 0) & (row < c["V"])
    out = st["table"][torch.where(live, row, torch.zeros_like(row))].float() * c["scale"]
    return torch.where(live[:, None], out, torch.zeros_like(out)).to(st["table"].dtype)


def _plain_embed_grad(st):
    c = st["case"]
    row = st["ids"].long() - c["first"]
    live = (row >= 0) & (row < c["V"])
    total = torch.zeros(c["V"] + 1, c["D"], device=DEV)
    total.index_add_(0, torch.where(live, row, torch.full_like(row, c["V"])), st["dy"].float())
    total = total[:c["V"]] * c["scale"]
    if c["accumulate"]:
        return st["grad"].copy_(st["grad"].float() + total)
    return total.to(_type(c["gdtype"]))


def _plain_clip(st):
    sums = torch.stack([v.float().square().sum() for v in st["grads"]])
    norm = sums.sum().sqrt()
    coef = (st["max_norm"] / (norm + EPS)).clamp(max=1.0)
    return {"norm": norm, "coef": coef, "out": (st["flat"].float() * coef).to(st["out"].dtype)}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_linear(st):
    from weight_communication_gb300 import fp8
    c = st["case"]
    w = fp8.Fp8Tensor(st["codes"], st["scales"], c["N"], c["K"], block_rows=BLOCK)
    x, _ = fp8.quantize(st["x"])
    return fp8.matmul(x, w)


def _own_train(st):
    from weight_communication_gb300 import fp8
    lin = fp8.Fp8Linear(st["w"])
    y, saved = lin.forward(st["x"], save=True)
    dx, dw = lin.backward(st["dy"], saved)
    return {"y": y, "dx": dx, "dw": dw}


def _own_embed(st):
    from weight_communication_gb300 import embedding
    c = st["case"]
    return embedding.lookup(st["table"], st["ids"], scale=c["scale"], first_row=c["first"])


def _own_embed_grad(st):
    from weight_communication_gb300 import embedding
    c = st["case"]
    if c["accumulate"]:
        return embedding.grad(st["dy"], st["ids"], c["V"], scale=c["scale"], first_row=c["first"],
                              out=st["grad"], accumulate=True)
    return embedding.grad(st["dy"], st["ids"], c["V"], scale=c["scale"], first_row=c["first"],
                          out_dtype=_type(c["gdtype"]))


def _own_clip(st):
    from weight_communication_gb300 import gradnorm
    stats = gradnorm.clip(st["list"], st["max_norm"], out=st["out_list"], eps=EPS)
    return {"norm": stats[0], "coef": stats[1], "out": st["out"]}


PLAIN = {"linear": _plain_linear, "train": _plain_train, "embed": _plain_embed,
         "embed_grad": _plain_embed_grad, "clip": _plain_clip}
OWN = {"linear": _own_linear, "train": _own_train, "embed": _own_embed,
       "embed_grad": _own_embed_grad, "clip": _own_clip}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def _size(name):
    return {"bf16": 2, "f32": 4}[name]


def work(case):
    op = case["op"]
    if op in ("linear", "train"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":
            return {"bytes": 2 * M * K + N * K + 4 * (-(-N // BLOCK)) * (-(-K // BLOCK)) + 2 * M * N,
                    "flops": 2 * M * N * K}
        return {"bytes": 2 * (M * K + N * K + M * N) + 2 * (M * N + M * K) + 4 * N * K,
                "flops": 6 * M * N * K}
    if op in ("embed", "embed_grad"):
        n, V, D = case["n"], case["V"], case["D"]
        e, i = _size(case["dtype"]), 8 if case["wide"] else 4
        hit = max(1, int(n * 0.98 * (0.71 if case["first"] else 1.0)))   # tokens with a row here
        rows = _expected_rows(hit, V)
        if op == "embed":
            return {"bytes": n * i + rows * D * e + n * D * e, "flops": hit * D}
        ge = _size(case["gdtype"])
        # adding touches the tokens' rows alone, a new gradient is written whole
        written = 2 * rows if case["accumulate"] else V
        return {"bytes": n * i + hit * D * e + written * D * ge, "flops": hit * D}
    n = sum(_spans(case))
    if case["inplace"] and not case["clipped"]:
        return {"bytes": n * _size(case["src"]), "flops": 2 * n}
    return {"bytes": n * (_size(case["src"]) + _size(case["dst"])), "flops": 3 * n}


def _expected_rows(hit, V):
    """Distinct rows among `hit` tokens of Zipf's law over V rows."""
    h, rows, k = math.log(V + 1), 0.0, 1
    while k <= V:                               # bands of ranks [k, 2k)
        top = min(2 * k, V + 1)
        p = math.log(top / k) / h / (top - k)
        rows += (top - k) * -math.expm1(-hit * p)
        k = top
    return max(1, int(rows))


def _exact_codes(v):
    """Nearest e4m3 values (ties to even) of v, by the spacing of its binade."""
    v = v.double()
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step).mul(step).clamp(-TOP, TOP)


def _exact_quantized(x, tall):
    """The 64-bit values that x (bf16 [R, C]) stands for, blocks of tall x 128.
    Which code a value gets is defined by one binary32 division and one
    binary32 product; all else is in 64 bits."""
    r, c = x.shape
    R, C = -(-r // tall) * tall, -(-c // BLOCK) * BLOCK
    p = torch.nn.functional.pad(x.float(), (0, C - c, 0, R - r))
    m = p.view(R // tall, tall, C // BLOCK, BLOCK).abs().amax(3).amax(1)
    dead = m < TOP * TINY
    inv = torch.full_like(m, TOP) / m.masked_fill(dead, 1.0)
    scale = (m / torch.full_like(m, TOP)).masked_fill(dead, 0.0)
    up = lambda t: t.repeat_interleave(tall, 0).repeat_interleave(BLOCK, 1)   # noqa: E731
    codes = _exact_codes(p * up(inv.masked_fill(dead, 0.0)))
    return (codes * up(scale).double())[:r, :c]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        N, K = case["N"], case["K"]
        s = st["scales"].double()
        at_n = torch.arange(N, device=DEV) // BLOCK
        at_k = torch.arange(K, device=DEV) // BLOCK
        w = st["codes"][:, :K].float().double() * s[at_k][:, at_n].t()
        return torch.einsum("mk,nk->mn", _exact_quantized(st["x"], 1), w)
    if op == "train":
        w = _exact_quantized(st["w"], BLOCK)
        y = torch.einsum("mk,nk->mn", _exact_quantized(st["x"], 1), w)
        dx = torch.einsum("mn,nk->mk", _exact_quantized(st["dy"], 1), w)
        dw = torch.einsum("nm,km->nk", _exact_quantized(st["dy"].t().contiguous(), 1),
                          _exact_quantized(st["x"].t().contiguous(), 1))
        return {"y": y, "dx": dx, "dw": dw}
    if op in ("embed", "embed_grad"):
        rows = st["ids"].long() - case["first"]
        here = ((rows >= 0) & (rows < case["V"])).nonzero()[:, 0]
        if op == "embed":
            out = torch.zeros(case["n"], case["D"], dtype=torch.float64, device=DEV)
            out[here] = st["table"].double()[rows[here]] * case["scale"]
            return out
        out = (st["grad"].double() if case["accumulate"] else
               torch.zeros(case["V"], case["D"], dtype=torch.float64, device=DEV))
        return out.index_put_((rows[here],), st["dy"].double()[here] * case["scale"],
                              accumulate=True)
    norm2 = torch.zeros((), dtype=torch.float64, device=DEV)
    for part in st["flat"].split(1 << 26):
        norm2 += torch.dot(part.double(), part.double())
    norm = norm2.sqrt()
    coef = torch.minimum(st["max_norm"] / (norm + EPS), torch.ones_like(norm))
    return {"norm": norm, "coef": coef,
            "out": None if case["inplace"] else st["flat"].double() * coef}
