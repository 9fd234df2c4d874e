"""One data-parallel training step with everything the package has, on one GPU.

    python -m weight_communication_gb300.train_step [--gated] [--ranks 4] [--steps 5] [...]

A small language model -- embedding, one residual 8-bit block and an 8-bit
output layer over the vocabulary -- is trained by simulated ranks that each
see their own tokens.  A step runs:

  1. on every rank: embedding lookup, 8-bit linear layers forward, the
     cross-entropy and its gradient (plain torch), 8-bit layers backward, and
     the embedding's gradient; all gradients land in the rank's row of one flat
     bf16 bucket;
  2. the qgZ reduce over the ranks (int4 with LoCo error feedback, average);
  3. the global norm of the reduced gradient and clipping;
  4. the update of fp32 master weights (momentum-free SGD, plain torch), and
     of the working weights: 8-bit for the layers, bf16 for the embedding.

`TrainStep` is the step as a class; the command prints the loss, the gradient
norm and the clipping coefficient of each step.

`GatedTrainStep` (--gated) is the same step with a larger block, and without the
plain torch of step 1: norm, gated 8-bit layers, residual sum, norm, and an output
layer whose loss and gradients come without logits.  Between forward and backward
it keeps activations and norm inputs in 8 bits.
"""
from __future__ import annotations

import argparse

import torch

from . import activation, embedding, fp8, gradnorm, loss, norm
from .qgz import QgzReducer


class TrainStep:
    """Weights, buffers and calls of the step.

    master  : fp32 [total], all parameters one after another, padded to what
              the reduce wants
    buckets : bf16 [ranks, total], every rank's gradient in the same order
    """

    def __init__(self, vocab: int, width: int, hidden: int, ranks: int = 4, lr: float = 0.2,
                 max_norm: float = 1.0, block: int = 256, seed: int = 0, device="cuda"):
        if width % 8 or hidden % 8:
            raise ValueError("width and hidden must be multiples of 8 (gradients start on 16 bytes)")
        self.vocab, self.width, self.ranks = vocab, width, ranks
        self.lr, self.max_norm, self.scale = lr, max_norm, float(width) ** 0.5
        self.shapes = self._shapes(vocab, width, hidden)
        count = sum(r * c for r, c in self.shapes.values())
        self.total = -(-count // (ranks * block)) * ranks * block
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.master = torch.zeros(self.total, device=device)
        self.weights = self._named(self.master)
        for name, w in self.weights.items():
            if w.shape[0] == 1:    # of a norm
                w.fill_(1.0)
                continue
            std = 1.0 / self.scale if name == "table" else w.shape[1] ** -0.5
            w.copy_(torch.randn(w.shape, generator=g, device=device) * std)
        self.bf16 = {n: self.weights[n].to(torch.bfloat16) for n in self.in_bf16}
        self.layers = {n: fp8.Fp8Linear(self.weights[n]) for n in self.in_8_bits}

        self.buckets = torch.zeros(ranks, self.total, dtype=torch.bfloat16, device=device)
        self.grads = [self._named(b) for b in self.buckets]
        self.reducer = QgzReducer(self.total, ranks, B=block, err_scale=1.0, err_beta=0.5,
                                  out_scale=1.0 / ranks, device=device)
        # the shards as the ranks own them: one list, named once
        self.shards = gradnorm.TensorList(self.reducer.out.view(ranks, -1).unbind())
        self.update = self._named(self.reducer.out)

    # working weights
    in_bf16, in_8_bits = ("table",), ("up", "down", "head")

    @staticmethod
    def _shapes(vocab: int, width: int, hidden: int) -> dict:
        return {"table": (vocab, width), "up": (hidden, width), "down": (width, hidden), "head": (vocab, width)}

    # (the step's parts by name)
    table = property(lambda self: self.bf16["table"])
    up = property(lambda self: self.layers["up"])
    down = property(lambda self: self.layers["down"])
    head = property(lambda self: self.layers["head"])

    def load(self) -> None:
        """The working weights from the master weights."""
        for name, w in self.bf16.items():
            w.copy_(self.weights[name])
        for name, lin in self.layers.items():
            lin.load(self.weights[name])

    def _named(self, flat: torch.Tensor) -> dict:
        out, at = {}, 0
        for name, (r, c) in self.shapes.items():
            out[name] = flat[at:at + r * c].view(r, c)
            at += r * c
        return out

    def rank_gradient(self, rank: int, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Forward and backward of one rank; fills its bucket, returns the loss."""
        grads = self.grads[rank]
        x = embedding.lookup(self.table, ids, self.scale)
        a, x_saved = self.up.forward(x, save=True)
        h = torch.relu(a)
        r, h_saved = self.down.forward(h, save=True)
        y = x + r
        logits, y_saved = self.head.forward(y, out_dtype=torch.float32, save=True)

        logp = torch.log_softmax(logits, dim=1)
        value = -logp.gather(1, targets[:, None]).mean()
        dlogits = logp.exp_()
        dlogits.scatter_add_(1, targets[:, None], torch.full_like(targets[:, None], -1.0, dtype=torch.float32))
        dlogits /= targets.numel()

        dy, _ = self.head.backward(dlogits, y_saved, dw=grads["head"])
        dh, _ = self.down.backward(dy, h_saved, dw=grads["down"])
        da = torch.where(a > 0, dh, torch.zeros_like(dh))
        dx, _ = self.up.backward(da, x_saved, dw=grads["up"])
        embedding.grad(dx + dy, ids, self.vocab, self.scale, out=grads["table"])
        return value

    def step(self, ids: torch.Tensor, targets: torch.Tensor):
        """ids, targets: [ranks, tokens].  Returns (mean loss, [norm, coef]) on
        the device; nothing waits for the GPU."""
        losses = [self.rank_gradient(r, ids[r], targets[r]) for r in range(self.ranks)]
        self.reducer.step(self.buckets)
        stats = gradnorm.clip(self.shards, self.max_norm)
        for name, w in self.weights.items():
            w.sub_(self.update[name], alpha=self.lr)
        self.load()
        return torch.stack(losses).mean(), stats


class GatedTrainStep(TrainStep):
    """The step of a model with one gated block between norms:

        n = norm(x),  y = x + down(silu(gate(n)) * up(n)),  loss of head(norm(y))
    """

    in_bf16, in_8_bits = ("table", "head", "norm_in", "norm_out"), ("gate", "up", "down")

    @staticmethod
    def _shapes(vocab: int, width: int, hidden: int) -> dict:
        return {"table": (vocab, width), "norm_in": (1, width), "gate": (hidden, width), "up": (hidden, width),
                "down": (width, hidden), "norm_out": (1, width), "head": (vocab, width)}

    def rank_gradient(self, rank: int, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        grads, w = self.grads[rank], self.bf16
        gate, up, down = (self.layers[n] for n in ("gate", "up", "down"))
        x = embedding.lookup(w["table"], ids, self.scale)
        n, _, kept_in = norm.rms(x, w["norm_in"][0], save=True)
        g = gate.forward(n)
        u, n_saved = up.forward(n, save=True)      # (the same for both layers)
        h, kept = activation.forward(g, u, kind="silu", save=True)
        r, h_saved = down.forward(h, save=True)
        z, _, kept_out = norm.rms(r, w["norm_out"][0], add=x, save=True)
        losses, lse = loss.cross_entropy(z, w["head"], targets, save=True)

        dz, _ = loss.cross_entropy_grad(z, w["head"], targets, lse, 1.0 / targets.numel(), dw=grads["head"])
        dy, _ = norm.rms_grad(dz, w["norm_out"][0], kept_out, dweight=grads["norm_out"][0])
        dh, _ = down.backward(dy, h_saved, dw=grads["down"])
        dg, du = activation.backward(dh, kept)
        dn, _ = gate.backward(dg, n_saved, dw=grads["gate"])
        dn_up, _ = up.backward(du, n_saved, dw=grads["up"])
        dx, _ = norm.rms_grad(dn + dn_up, w["norm_in"][0], kept_in, add=dy, dweight=grads["norm_in"][0])
        embedding.grad(dx, ids, self.vocab, self.scale, out=grads["table"])
        return losses.mean()


def batch(vocab: int, ranks: int, tokens: int, step: int, device="cuda"):
    """Synthetic text: each token is followed by a fixed function of it."""
    g = torch.Generator(device=device)
    g.manual_seed(1000 + step)
    ids = torch.randint(0, vocab, (ranks, tokens), generator=g, device=device)
    return ids, (ids * 7 + 3) % vocab


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=688)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=2048, help="per rank and step")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--gated", action="store_true", help="the gated block between norms, and the loss without logits")
    args = ap.parse_args(argv)
    model = (GatedTrainStep if args.gated else TrainStep)(args.vocab, args.width, args.hidden, args.ranks)
    rows = []
    for i in range(args.steps):
        ids, targets = batch(args.vocab, args.ranks, args.tokens, i)
        rows.append(model.step(ids, targets))
    for i, (value, stats) in enumerate(rows):
        length, coef = stats.tolist()
        print(f"step {i}: loss {float(value):.4f}, gradient norm {length:.4f}, coefficient {coef:.4f}")


if __name__ == "__main__":
    main()
