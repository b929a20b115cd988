"""How many digits fp32 products of bf16 parts keep: rms errors, and the products as their parts say.

Worst cases over a sum leave room for a lost part, 2^-17 of a value.  The rms
over a matrix of random elements does not.  U is half a step of fp32.

A sum's parts are added smallest first, so that only the products of first parts
meet a running sum of the result's size: k / 32 + 1 matrix instructions of 32
products each, and a tenth more for the parts before.  Where a tile's steps of 64
are cut, stretches of at least four (of six parts' steps) are added, 1.5 (k / 64 + 1)
at most.  Each rounding is at most a whole step, 2 U, of a running sum whose size
is on average 1 / sqrt(2) of the result's.  Even if all roundings go one way, a
result is off by
    sqrt(2) U (1.1 (k / 32 + 1) + 1.5 (k / 64 + 1))
of its size, and by 2.1 U for the parts' products that are left out.  dx is the sum
of two such products; all six parts of the second one's meet the first one's sum.
Errors of operands are of either sign in a product's terms: they add up as squares.
"""
import math

import torch

import step_oracle as so

U = so.U


def sums(k, both=False):
    n = k / 32 + 1
    return math.sqrt(2) * U * (1.1 * n + 1.5 * (k / 64 + 1) * (2 if both else 1) + (6 * n if both else 0)) + 2.1 * U


def rms(x):
    return x.double().square().mean().sqrt().item()


def off(got, ref):
    """rms of the error, relative to the values'."""
    return rms(got.double().cpu() - ref.double().cpu()) / rms(ref)


def split(v, count):
    """v as bf16 values, each of what those before it left."""
    out = []
    v = v.double()
    for _ in range(count):
        out.append(v.to(torch.bfloat16).double())
        v = v - out[-1]
    return out


SEGMENTS = [(0, 0), (0, 1), (1, 0), (0, 2), (1, 1), (2, 0)]


def product(a, b, segments):
    """a @ b.T as the products of parts (i, j) of the two, rounded to fp32 once."""
    pa, pb = split(a, 3), split(b, 3)
    return sum(pa[i] @ pb[j].t() for i, j in segments).float()


# ------------------------------------------------------------ feed-forward
def one_a_row(m, g, low=-3, high=4):
    """m with all but one element of each row 0, which is a power of two: its products have one term and are exact."""
    at = torch.randint(0, m.shape[1], (m.shape[0], 1), generator=g)
    return torch.zeros_like(m).scatter_(1, at, 2.0 ** torch.randint(low, high, at.shape, generator=g))


def block_inputs(rows, dim, hidden, names):
    """x, w_gate, w_up, w_down, dout, and gate and up for the gradients: dense but for those whose products only lead to
    the ones looked at."""
    g = torch.Generator().manual_seed(rows + dim + hidden)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, wg, wu, wd, dy = (rand(rows, dim), rand(hidden, dim) / dim ** 0.5, rand(hidden, dim) / dim ** 0.5, rand(dim, hidden) / hidden ** 0.5,
                         rand(rows, dim))
    if "out" in names:
        x = one_a_row(x, g)
    if "dx" in names:
        dy = one_a_row(dy, g)
    if "dw_up" in names:
        wd = one_a_row(wd.t(), g).t().contiguous()
    return x, wg, wu, wd, dy, rand(rows, hidden), rand(rows, hidden)


def block(x, wg, wu, wd, dy, gate, up, names, segments=None):
    """The named results of the block with relu, in 64 bits or of parts."""
    if segments is None:
        x, wg, wu, wd, dy, gate, up = (m.double() for m in (x, wg, wu, wd, dy, gate, up))
        mul = lambda a, b: a @ b.t()  # noqa: E731
    else:
        mul = lambda a, b: product(a, b, segments)  # noqa: E731
    out = {}
    if "gate" in names or "out" in names:
        own = mul(x, wg), mul(x, wu)
        out["gate"], out["up"] = own
    if "out" in names:
        out["out"] = mul(own[0].clamp(min=0) * own[1], wd)
    if "dx" in names or "dw_up" in names:
        act = gate.clamp(min=0)
        s, ds = act * up, mul(dy, wd.t())
        dg, du = ds * up * (gate > 0), ds * act
    if "dx" in names:
        out["dx"] = mul(torch.cat([dg, du], 1), torch.cat([wg, wu]).t())
    if "dw_up" in names:
        out["dw_gate"], out["dw_up"], out["dw_down"] = mul(dg.t(), x.t()), mul(du.t(), x.t()), mul(dy.t(), s.t())
    return {n: out[n] for n in names}


def block_bounds(rows, dim, hidden):
    """Of those results; the roundings of an operand made in an epilogue (two or three products) are 4 U."""
    return {"gate": sums(dim), "up": sums(dim), "out": math.hypot(4 * U, sums(hidden)), "dx": math.hypot(4 * U, sums(hidden, True)),
            "dw_gate": math.hypot(4 * U, sums(rows)), "dw_up": math.hypot(4 * U, sums(rows)), "dw_down": math.hypot(4 * U, sums(rows))}


# Each with the results whose sums are short enough to tell two parts from three.
BLOCKS = [
    (200, 64, 264, ("gate", "up")), (2200, 64, 2400, ("gate", "up")), (700, 96, 1100, ("gate", "up")),
    (200, 264, 32, ("out", "dx")), (2200, 2304, 32, ("out", "dx")), (1100, 700, 48, ("out", "dx")), (700, 1100, 96, ("out",)),
    (66, 264, 200, ("dw_gate", "dw_up", "dw_down")), (66, 2304, 2400, ("dw_gate", "dw_up", "dw_down")),
    (80, 700, 1100, ("dw_gate", "dw_up", "dw_down")), (4000, 4096, 32, ("out", "dx")),  # (large tiles)
    (200, 256, 264, ("gate", "up")), (200, 264, 256, ("out",)), (256, 264, 200, ("dw_gate", "dw_up", "dw_down")),  # (cut ones)
]


# ------------------------------- log probabilities from the hidden state
def head_inputs(rows, vocab, dim, name):
    """hidden, weight, tokens, dlogprob, dentropy.  For gradients the logits are exact, and those of the entropy alone:
    a row's dz has no element that outweighs the others."""
    g = torch.Generator().manual_seed(rows + vocab + dim)
    h, w = torch.randn(rows, dim, generator=g), torch.randn(vocab, dim, generator=g)
    tok = torch.randint(0, vocab, (rows,), generator=g)
    if name == "logprob":
        return h, w * (64 / dim ** 0.5), tok, None, None
    if name == "dhidden":
        h = one_a_row(h, g, -1, 1)
    else:
        w = one_a_row(w, g, -1, 1)
    return h, w, torch.full_like(tok, -1), torch.zeros(rows), torch.randn(rows, generator=g)


def head(h, w, tok, gl, ge, name, segments=None):
    """logprob, dhidden or dweight, in 64 bits or of parts."""
    mul = (lambda a, b: a @ b.t()) if segments is None else (lambda a, b: product(a, b, segments).double())
    h, w = h.double(), w.double()
    logp = torch.log_softmax(mul(h, w), 1)
    if name == "logprob":
        return logp.gather(1, tok[:, None])[:, 0]
    p = logp.exp()
    dz = -ge.double()[:, None] * p * (logp - (p * logp).sum(1, keepdim=True))
    return mul(dz, w.t()) if name == "dhidden" else mul(dz.t(), h.t())


def head_bounds(rows, vocab, dim):
    """The logprob's is relative to the logits' size, 64: a logit less the log of a sum, both with the product's error and
    of up to 7 times that size, in three roundings.  Of dz, log p is below 16 and rounded three times (8 U each), its exponential is off by as much
    and 2 U, log p + entropy, which is about 1, by as much again: 20 U in squares, as either sign is as likely."""
    return {"logprob": math.hypot(sums(dim), sums(dim), 3 * 7 * U), "dhidden": math.hypot(20 * U, sums(vocab)),
            "dweight": math.hypot(20 * U, sums(rows))}


def head_off(name, got, ref):
    return rms(got.double().cpu() - ref) / 64 if name == "logprob" else off(got, ref)


HEADS = [(100, 300, 64, "logprob"), (2200, 2400, 64, "logprob"), (1100, 700, 96, "logprob"), (200, 96, 264, "dhidden"),
         (2200, 64, 2304, "dhidden"), (66, 264, 200, "dweight"), (66, 2400, 2304, "dweight"), (96, 700, 1100, "dweight"),
         (300, 400, 250, "logprob")]
