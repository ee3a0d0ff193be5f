"""A small language model trained end to end with the library.

``python -m rank_gradient_sketching_philox_gb300.train_example``

Embedding -> blocks of x + W2 relu(W1 norm(x)) -> norm -> linear head.  Every
linear layer, the head too, is trained by its gradient sketch: it saves the
projected input XP, accumulates C += D^T XP and is updated by normalized SGD with
stochastic rounding.  The layer norms make the sketched layers' inputs, the cross
entropy starts the backward pass over the head's vocabulary without its logits and
hands the head's sketch over in the same call, and AdamW with 8-bit states updates
what is not sketched: the embedding, the norms' weights and biases.

The matrix products of the forward pass and of the input gradients, the embedding's
lookup and the additions between the layers are plain torch.
"""
import argparse

import torch

from . import binding as rgs
from .optimizer import AdamW

BF, F32 = torch.bfloat16, torch.float32


class Linear:
    """A sketched linear layer: W (d x k BF16), its sketch C and this step's projection P."""

    def __init__(self, d, k, r, layer, gen, dev):
        self.W = (torch.randn(d, k, generator=gen, device=dev) * k ** -0.5).to(BF)
        self.C = torch.zeros(d, r, device=dev)
        self.P = torch.empty(k, r, device=dev)
        self.XP = None
        self.layer = layer

    def save(self, X):
        """Keep X P for the backward pass, instead of X."""
        self.XP = torch.empty(X.shape[0], self.P.shape[1], dtype=BF, device=X.device)
        rgs.project_inputs(X, self.P, self.XP)

    def forward(self, X):
        self.save(X)
        return X @ self.W.t()

    def backward(self, D, overwrite):
        rgs.accumulate(D, self.XP, self.C, overwrite=overwrite)
        return D @ self.W


class Norm:
    def __init__(self, k, dev):
        self.gamma, self.beta = torch.ones(k, dtype=BF, device=dev), torch.zeros(k, dtype=BF, device=dev)
        self.dgamma, self.dbeta = torch.zeros(k, device=dev), torch.zeros(k, device=dev)

    def forward(self, X):
        T, dev = X.shape[0], X.device
        self.X, Y = X, torch.empty_like(X)
        self.mean, self.rstd = torch.empty(T, device=dev), torch.empty(T, device=dev)
        return rgs.layer_norm_forward(X, self.gamma, self.beta, Y, self.mean, self.rstd)

    def backward(self, dY, overwrite):
        return rgs.layer_norm_backward(dY, self.X, self.gamma, self.mean, self.rstd, torch.empty_like(dY), self.dgamma,
                                       self.dbeta, overwrite=overwrite)


class Model:
    def __init__(self, vocabulary=1000, width=256, blocks=2, rank=64, tau=0.02, lr=2e-3, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.tau, self.lr, self.rank, self.seed, self.count = tau, lr, rank, seed, 0
        self.norms = [Norm(width, device) for _ in range(blocks + 1)]
        self.pairs = [(Linear(4 * width, width, rank, 2 * b, gen, device), Linear(width, 4 * width, rank, 2 * b + 1, gen, device))
                      for b in range(blocks)]
        self.head = Linear(vocabulary, width, rank, 2 * blocks, gen, device)
        self.linears = [layer for pair in self.pairs for layer in pair] + [self.head]
        self.embedding = torch.randn(vocabulary, width, generator=gen, device=device).to(BF)
        self.dembedding = torch.zeros(vocabulary, width, device=device)
        params = [self.embedding] + [w for n in self.norms for w in (n.gamma, n.beta)]
        grads = [self.dembedding] + [g for n in self.norms for g in (n.dgamma, n.dbeta)]
        self.adam = AdamW(params, grads, state_bits=8, seed=seed, layers=range(1000, 1000 + len(params)))

    def microbatch(self, tokens, targets, first, weight):
        """Forward and backward of one microbatch; returns its tokens' losses.  A negative target is ignored."""
        dev = tokens.device
        x = self.embedding[tokens]
        for norm, (up, down) in zip(self.norms, self.pairs):
            h = torch.relu(up.forward(norm.forward(x)))
            up.active = h > 0
            x = x + down.forward(h)
        y = self.norms[-1].forward(x)
        self.head.save(y)
        loss, lse = torch.empty(len(tokens), device=dev), torch.empty(len(tokens), device=dev)
        rgs.cross_entropy_forward(y, self.head.W, targets, loss, lse)
        g = torch.full((len(tokens),), weight, device=dev)
        dx = torch.empty_like(y)
        rgs.cross_entropy_backward(y, self.head.W, targets, lse, g, dX=dx, XP=self.head.XP, C=self.head.C,
                                   overwrite=first)
        dx = self.norms[-1].backward(dx, first)
        for norm, (up, down) in zip(reversed(self.norms[:-1]), reversed(self.pairs)):
            dh = torch.where(up.active, down.backward(dx, first), 0.0)
            dx = dx + norm.backward(up.backward(dh, first), first)
        if first:
            self.dembedding.zero_()
        self.dembedding.index_add_(0, tokens, dx.float())
        return loss

    def step(self, microbatches):
        """One training step over (tokens, targets) pairs; returns the mean loss of the tokens that count."""
        rgs.sample_projection_batched(rgs.PROJ_GAUSSIAN_QR, self.seed, self.count, [m.P for m in self.linears[:-1]],
                                      [m.layer for m in self.linears[:-1]])
        rgs.sample_projection(rgs.PROJ_GAUSSIAN_QR, self.seed, self.head.layer, self.count, self.head.P)
        kept = sum(int((t >= 0).sum()) for _, t in microbatches)
        losses = [self.microbatch(x, t, i == 0, 1.0 / kept) for i, (x, t) in enumerate(microbatches)]
        rgs.apply_update_normsgd_batched([m.W for m in self.linears], [m.C for m in self.linears],
                                         [m.P for m in self.linears], self.tau, self.seed,
                                         [m.layer for m in self.linears], self.count)
        self.adam.step(self.lr, self.count)
        self.count += 1
        return torch.cat(losses).sum() / kept


def task(vocabulary, tokens, microbatches, step, device="cuda"):
    """Successors under a fixed permutation, a tenth of them ignored."""
    gen = torch.Generator(device=device).manual_seed(17)
    successor = torch.randperm(vocabulary, generator=gen, device=device)
    gen.manual_seed(1000 + step)
    out = []
    for _ in range(microbatches):
        x = torch.randint(0, vocabulary, (tokens,), generator=gen, device=device)
        ignored = torch.rand(tokens, generator=gen, device=device) < 0.1
        out.append((x, torch.where(ignored, -1, successor[x])))
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--vocabulary", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args(argv)
    model = Model(a.vocabulary, a.width, a.blocks)
    losses = []
    for step in range(a.steps):
        losses.append(float(model.step(task(a.vocabulary, a.tokens, 2, step))))
        if step % 10 == 0 or step == a.steps - 1:
            print("step %4d  loss %.4f" % (step, losses[-1]))
    return losses


if __name__ == "__main__":
    main()
