"""A training step whose matrix products are the package's too: embedding, layer
norm, a gated feed-forward block beside a residual, and the next tokens' log
probabilities straight from the hidden state, with all their gradients.

As in ``train_step.py``, W ranks on one GPU have a batch each and one
tensor-fusion all-reduce averages the gradients; then the block's three matrices
move by the orthogonalised running mean of theirs, the others by its sign.

    python examples/train_block.py --steps 40
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_reduction_ring_amd as rsx  # noqa: E402


class Rank:
    """One rank's parameters and gradients (fp32), activations (of ``dtype``) and plans."""

    NAMES = ("table", "weight", "bias", "proj", "w_gate", "w_up", "w_down")

    def __init__(self, vocab: int, dim: int, hidden: int, tokens: int, seed: int, dtype=torch.bfloat16):
        dev = "cuda:0"
        g = torch.Generator(device=dev).manual_seed(7)  # the same parameters on every rank
        rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.params = [rand(vocab, dim) * 0.1, torch.ones(dim, device=dev), torch.zeros(dim, device=dev), rand(vocab, dim) * 0.1,
                       rand(hidden, dim) / dim ** 0.5, rand(hidden, dim) / dim ** 0.5, rand(dim, hidden) / hidden ** 0.5]
        self.grads = [torch.empty_like(p) for p in self.params]
        table, weight, bias, proj, *block = self.params
        self.low = [p.to(dtype) for p in (proj, *block)]  # what is multiplied
        self.data = torch.Generator(device=dev).manual_seed(seed)
        self.vocab = vocab

        # forward
        self.tokens = torch.zeros(tokens, dtype=torch.int64, device=dev)
        self.targets = torch.zeros_like(self.tokens)
        x = torch.empty(tokens, dim, dtype=dtype, device=dev)
        self.embed = rsx.Embedding(table, self.tokens, x, scale=dim ** 0.5)
        self.norm = rsx.LayerNorm(x, weight, bias)
        self.block = rsx.FeedForward(self.norm.out, *self.low[1:], keep=True)
        self.x, self.sum = x, torch.empty_like(x)
        self.logp = rsx.LinearLogprobs(self.sum, self.low[0], self.targets, scale=dim ** -0.5)
        # backward of the mean of -log p
        minus = torch.full((tokens,), -1.0 / tokens, device=dev)
        self.dlogp = rsx.LinearLogprobsGrad(self.sum, self.low[0], self.targets, self.logp.lse, minus, dweight=self.grads[3],
                                            lse_rest=self.logp.lse_rest, scale=dim ** -0.5)
        self.dblock = rsx.FeedForwardGrad(self.dlogp.dhidden, self.norm.out, *self.low[1:], self.block.gate, self.block.up, None,
                                          *self.grads[4:])
        self.dnorm = rsx.LayerNormGrad(self.dblock.dx, x, self.norm.mean, self.norm.rstd, weight, dx=self.dblock.dx,
                                       dweight=self.grads[1], dbias=self.grads[2])
        self.dembed = rsx.EmbeddingGrad(self.dblock.dx, self.tokens, self.grads[0], scale=dim ** 0.5)

    def next_batch(self) -> None:
        """Tokens, each followed by a fixed other one: what the model can learn."""
        self.tokens.random_(0, self.vocab, generator=self.data)
        torch.remainder(self.tokens * 5 + 3, self.vocab, out=self.targets)

    def gradients(self) -> torch.Tensor:
        """The batch's loss; its gradients go to self.grads."""
        for low, p in zip(self.low, self.params[3:]):
            low.copy_(p)
        self.embed()
        self.norm()
        self.block()
        torch.add(self.x, self.block.out, out=self.sum)
        self.logp()
        self.dlogp()
        self.dblock()
        self.dnorm()
        self.dblock.dx.add_(self.dlogp.dhidden)  # the residual's
        self.dembed()
        return -self.logp.logprob.mean()


class Updates:
    """One rank's steps: by the sign of the gradients' running mean, or by that mean orthogonalised."""

    def __init__(self, rank: Rank, rate: float):
        self.rank, self.rate = rank, rate
        self.means = [torch.zeros_like(p) for p in rank.params]
        self.orthogonal = [rsx.NewtonSchulz(m) for m in self.means[4:]]

    def __call__(self) -> None:
        for p, g, m in zip(self.rank.params, self.rank.grads, self.means):
            m.mul_(0.9).add_(g, alpha=0.1)
        for p, m in zip(self.rank.params[:4], self.means):
            p.add_(m.sign(), alpha=-self.rate * 0.1)
        for p, o in zip(self.rank.params[4:], self.orthogonal):
            o()
            p.add_(o.out, alpha=-self.rate * max(1.0, p.shape[0] / p.shape[1]) ** 0.5)


def train(ranks: int = 4, steps: int = 40, vocab: int = 1000, dim: int = 256, hidden: int = 512, tokens: int = 2048, rate: float = 0.05):
    """(losses by step, the ranks)."""
    world = [Rank(vocab, dim, hidden, tokens, seed=r) for r in range(ranks)]
    reduce = rsx.TensorFusionAllReduce([r.grads for r in world], None, "avg")
    updates = [Updates(r, rate) for r in world]
    losses = []
    for _ in range(steps):
        total = 0.0
        for r in world:
            r.next_batch()
            total = total + r.gradients()
        reduce()
        for u in updates:
            u()
        losses.append((total / ranks).item())
    return losses, world


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    losses, world = train(a.ranks, a.steps, a.vocab, a.dim, a.hidden, a.tokens)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.4f}")
    same = all(torch.equal(p, q) for r in world[1:] for p, q in zip(r.params, world[0].params))
    print("parameters equal on all ranks:", same)


if __name__ == "__main__":
    main()
