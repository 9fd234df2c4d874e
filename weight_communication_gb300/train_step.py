"""One data-parallel training step with everything the package has, on one GPU.

    python -m weight_communication_gb300.train_step [--ranks 4] [--steps 5] [...]

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
"""
from __future__ import annotations

import argparse

import torch

from . import embedding, fp8, gradnorm
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
        self.shapes = {"table": (vocab, width), "up": (hidden, width), "down": (width, hidden),
                       "head": (vocab, width)}
        count = sum(r * c for r, c in self.shapes.values())
        self.total = -(-count // (ranks * block)) * ranks * block
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.master = torch.zeros(self.total, device=device)
        self.weights = self._named(self.master)
        for name, w in self.weights.items():
            std = 1.0 / self.scale if name == "table" else w.shape[1] ** -0.5
            w.copy_(torch.randn(w.shape, generator=g, device=device) * std)
        self.table = self.weights["table"].to(torch.bfloat16)
        self.up, self.down, self.head = (fp8.Fp8Linear(self.weights[n]) for n in ("up", "down", "head"))

        self.buckets = torch.zeros(ranks, self.total, dtype=torch.bfloat16, device=device)
        self.grads = [self._named(b) for b in self.buckets]
        self.reducer = QgzReducer(self.total, ranks, B=block, err_scale=1.0, err_beta=0.5,
                                  out_scale=1.0 / ranks, device=device)
        # the shards as the ranks own them: one list, named once
        self.shards = gradnorm.TensorList(self.reducer.out.view(ranks, -1).unbind())
        self.update = self._named(self.reducer.out)

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
        loss = -logp.gather(1, targets[:, None]).mean()
        dlogits = logp.exp_()
        dlogits.scatter_add_(1, targets[:, None], torch.full_like(targets[:, None], -1.0, dtype=torch.float32))
        dlogits /= targets.numel()

        dy, _ = self.head.backward(dlogits, y_saved, dw=grads["head"])
        dh, _ = self.down.backward(dy, h_saved, dw=grads["down"])
        da = torch.where(a > 0, dh, torch.zeros_like(dh))
        dx, _ = self.up.backward(da, x_saved, dw=grads["up"])
        embedding.grad(dx + dy, ids, self.vocab, self.scale, out=grads["table"])
        return loss

    def step(self, ids: torch.Tensor, targets: torch.Tensor):
        """ids, targets: [ranks, tokens].  Returns (mean loss, [norm, coef]) on
        the device; nothing waits for the GPU."""
        losses = [self.rank_gradient(r, ids[r], targets[r]) for r in range(self.ranks)]
        self.reducer.step(self.buckets)
        stats = gradnorm.clip(self.shards, self.max_norm)
        for name, w in self.weights.items():
            w.sub_(self.update[name], alpha=self.lr)
        self.table.copy_(self.weights["table"])
        for name, lin in (("up", self.up), ("down", self.down), ("head", self.head)):
            lin.load(self.weights[name])
        return torch.stack(losses).mean(), stats


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
    args = ap.parse_args(argv)
    model = TrainStep(args.vocab, args.width, args.hidden, args.ranks)
    rows = []
    for i in range(args.steps):
        ids, targets = batch(args.vocab, args.ranks, args.tokens, i)
        rows.append(model.step(ids, targets))
    for i, (loss, stats) in enumerate(rows):
        norm, coef = stats.tolist()
        print(f"step {i}: loss {float(loss):.4f}, gradient norm {norm:.4f}, coefficient {coef:.4f}")


if __name__ == "__main__":
    main()
