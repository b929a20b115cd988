"""Data-parallel training of a small language model on one GPU: the operators
make the gradients, the ring all-reduce averages them.

Each of W ranks (buffers on one GPU) has a batch of its own: embedding lookup,
a layer norm that keeps its input in 8 bits, a product with the output matrix,
the log probabilities of the next tokens.  Backward, the norm reads the 8-bit
input, the table's gradient is summed by sorted tokens, and one tensor-fusion
all-reduce averages all gradients.  Every call is a plan, made once.

    python examples/train_step.py --steps 40
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_reduction_ring_amd as rsx  # noqa: E402


class Rank:
    """One rank's parameters (fp32), activations (bf16) and plans."""

    def __init__(self, vocab: int, dim: int, tokens: int, seed: int):
        dev = "cuda:0"
        g = torch.Generator(device=dev).manual_seed(7)  # the same parameters on every rank
        self.table = torch.randn(vocab, dim, generator=g, device=dev) * 0.1
        self.weight, self.bias = torch.ones(dim, device=dev), torch.zeros(dim, device=dev)
        self.proj = torch.randn(vocab, dim, generator=g, device=dev) * 0.1
        self.params = [self.table, self.weight, self.bias, self.proj]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.proj16 = self.proj.bfloat16()
        self.data = torch.Generator(device=dev).manual_seed(seed)
        self.vocab = vocab

        # forward
        self.tokens = torch.zeros(tokens, dtype=torch.int64, device=dev)
        self.targets = torch.zeros_like(self.tokens)
        x = torch.empty(tokens, dim, dtype=torch.bfloat16, device=dev)
        self.embed = rsx.Embedding(self.table, self.tokens, x, scale=dim ** 0.5)
        self.norm = rsx.LayerNorm(x, self.weight, self.bias, checkpoint=rsx.Checkpoint(x.shape, dev))
        self.logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device=dev)
        self.logp = rsx.TokenLogprobs(self.logits, self.targets)
        # backward of the mean of -log p; the logits' gradient takes their place
        minus = torch.full((tokens,), -1.0 / tokens, device=dev)
        self.dlogits = rsx.TokenLogprobsGrad(self.logits, self.targets, self.logp.lse, minus, dlogits=self.logits,
                                             lse_rest=self.logp.lse_rest)
        self.dy = torch.empty_like(x)
        self.dnorm = rsx.LayerNormGrad(self.dy, self.norm.checkpoint, self.norm.mean, self.norm.rstd, self.weight, dx=self.dy,
                                       dweight=self.grads[1], dbias=self.grads[2])
        self.dembed = rsx.EmbeddingGrad(self.dy, self.tokens, self.grads[0], scale=dim ** 0.5)

    def next_batch(self) -> None:
        """Tokens, each followed by a fixed other one: what the model can learn."""
        self.tokens.random_(0, self.vocab, generator=self.data)
        torch.remainder(self.tokens * 5 + 3, self.vocab, out=self.targets)

    def gradients(self) -> torch.Tensor:
        """The batch's loss; its gradients go to self.grads."""
        self.proj16.copy_(self.proj)
        self.embed()
        self.norm()
        torch.mm(self.norm.out, self.proj16.t(), out=self.logits)
        self.logp()
        self.dlogits()
        self.grads[3].copy_(torch.mm(self.logits.t(), self.norm.out))
        torch.mm(self.logits, self.proj16, out=self.dy)
        self.dnorm()
        self.dembed()
        return -self.logp.logprob.mean()


def train(ranks: int = 4, steps: int = 40, vocab: int = 1000, dim: int = 256, tokens: int = 2048, rate: float = 0.05):
    """(losses by step, the ranks)."""
    world = [Rank(vocab, dim, tokens, seed=r) for r in range(ranks)]
    reduce = rsx.TensorFusionAllReduce([r.grads for r in world], None, "avg")
    moments = [[torch.zeros_like(p) for p in r.params] for r in world]
    losses = []
    for _ in range(steps):
        total = 0.0
        for r in world:
            r.next_batch()
            total = total + r.gradients()
        reduce()
        for r, ms in zip(world, moments):
            for p, g, m in zip(r.params, r.grads, ms):
                # steps of one size, by the sign of the gradients' running mean
                m.mul_(0.9).add_(g.sign(), alpha=0.1)
                p.add_(m.sign(), alpha=-rate * 0.1)
        losses.append((total / ranks).item())
    return losses, world


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    losses, world = train(a.ranks, a.steps, a.vocab, a.dim, a.tokens)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.4f}")
    same = all(torch.equal(p, q) for r in world[1:] for p, q in zip(r.params, world[0].params))
    print("parameters equal on all ranks:", same)
    # serving: the likeliest next tokens of a few, with their log probabilities
    r = world[0]
    lp = rsx.token_logprobs(torch.mm(rsx.layer_norm(rsx.embedding(r.table, r.tokens[:3], scale=a.dim ** 0.5), r.weight, r.bias)[0],
                                     r.proj.t()), r.targets[:3], top=2)
    for i in range(3):
        print(f"after {r.tokens[i].item()}: {lp.top_token[i].tolist()} {[round(v, 3) for v in lp.top_logprob[i].tolist()]}"
              f" (right: {r.targets[i].item()}), entropy {lp.entropy[i].item():.3f}")


if __name__ == "__main__":
    main()
