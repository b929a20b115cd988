"""The step's matrix products from their definitions, in 64 bits, with bounds on what a kernel may differ by.

U is half a step of fp32.  A sum of n products in fp32 in any order is off by at
most n * 2 U times the sum of their magnitudes: the matrix instructions' order
is not known, nor whether each addition rounds to nearest, so a whole step is
counted for each.  16-bit operands have exact products.  An fp32 value is the sum
of three bf16 values, each at most 2^-8 of the one before: of its products those
of parts (1,2), (2,1) and (2,2) are left out, less than 2.1 U of the product,
and the others are 6 n terms whose magnitudes add up to at most 1.02 times the
product's.
"""
import math

import torch

import step_oracle as so

U = so.U


def terms(dtype, k, parts=None):
    """The bound of a sum of k products, as a multiple of the sum of their magnitudes."""
    n = {1: 1, 2: 3, 3: 6}[(3 if dtype == torch.float32 else 1) if parts is None else parts]
    left_out = {1: 0.0, 3: 3 * 2.0 ** -16, 6: 2.1 * U}[n]  # of two parts of bf16, the product of the second ones
    return 1.02 * (n * k + 8) * 2 * U + left_out


def kept(dtype):
    """What rounding an operand to its type costs; fp32 is kept whole."""
    return 0.0 if dtype == torch.float32 else so.half(dtype)


# ------------------------------------------------------------ feed-forward
def activation(name, x):
    """(act, its slope) in x's 64 bits."""
    if name == "relu":
        return x.clamp(min=0), (x > 0).double()
    if name == "silu":
        p = torch.sigmoid(x)
        return x * p, p + x * p * (1 - p)
    if name == "gelu":
        p = 0.5 * torch.erfc(-x * math.sqrt(0.5))
        return x * p, p + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * c * (x + 0.044715 * x ** 3))
    return x * p, p + x * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * x * x)


SLOPE = 1.2    # the largest slope of any of them
BEND = 1.2     # and of the slopes'
EVAL = 64 * U  # an activation or slope in fp32: a few steps of exp or erfc and of the products, their argument's rounding included


def feed_forward(x, wg, wu, wd, act):
    """((y, g, u), bounds without the last rounding); x (rows, dim)."""
    t = x.dtype
    x, wg, wu, wd = (v.double() for v in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    k = terms(t, x.shape[1])
    eg, eu = k * (x.abs() @ wg.abs().t()), k * (x.abs() @ wu.abs().t())
    a, _ = activation(act, g)
    s = a * u
    ea = SLOPE * eg + EVAL * g.abs() * (1 + g.abs())
    es = ea * (u.abs() + eu) + a.abs() * eu + 2 * U * s.abs()
    es = es + kept(t) * (s.abs() + es)
    y = s @ wd.t()
    ey = es @ wd.abs().t() + terms(t, s.shape[1]) * ((s.abs() + es) @ wd.abs().t())
    if t == torch.float16:  # s below fp16's smallest normal keeps half of its smallest step
        ey = ey + 2.0 ** -25 * wd.abs().sum(1)
    return (y, g, u), (ey, eg, eu)


def feed_forward_grad(dy, x, wg, wu, wd, gate, up, act):
    """((dx, dwg, dwu, dwd), bounds without the last rounding), for gate and up as given."""
    t = x.dtype
    dy, x, wg, wu, wd, g, u = (v.double() for v in (dy, x, wg, wu, wd, gate, up))
    a, slope = activation(act, g)
    ea = EVAL * (1 + g.abs()) * (1 + g.abs())
    ds = dy @ wd
    eds = terms(t, dy.shape[1]) * (dy.abs() @ wd.abs())
    s, dg, du = a * u, ds * u * slope, ds * a
    small = 2.0 ** -25 if t == torch.float16 else 0.0

    def rounded(v, e):
        e = e + 4 * U * v.abs()
        return e + kept(t) * (v.abs() + e) + small
    es = rounded(s, ea * u.abs())
    edg = rounded(dg, (eds * slope.abs() + (ds.abs() + eds) * ea) * u.abs())
    edu = rounded(du, eds * a.abs() + (ds.abs() + eds) * ea)

    def product(p, ep, q):
        return p @ q, ep @ q.abs() + terms(t, p.shape[1]) * ((p.abs() + ep) @ q.abs())
    dx1, e1 = product(dg, edg, wg)
    dx2, e2 = product(du, edu, wu)
    dx, ex = dx1 + dx2, 2 * (e1 + e2)  # one sum of twice the length
    dwg, eg = product(dg.t(), edg.t(), x)
    dwu, eu = product(du.t(), edu.t(), x)
    dwd_t, ed = product(s.t(), es.t(), dy)
    return (dx, dwg, dwu, dwd_t.t()), (ex, eg, eu, ed.t())


# ------------------------------- log probabilities from the hidden state
def logits(hidden, weight, scale):
    """(z, bound)."""
    h, w = hidden.double(), weight.double()
    scale = float(torch.tensor(scale, dtype=torch.float32))
    z = scale * (h @ w.t())
    return z, abs(scale) * terms(hidden.dtype, h.shape[1]) * (h.abs() @ w.abs().t()) + U * z.abs()


def linear_logprobs(hidden, weight, tokens, scale):
    """(results, bounds): those of the exact logits, and what the logits' errors make of them."""
    z, ez = logits(hidden, weight, scale)
    out, tol = so.token_logprobs(z, tokens, 0)
    worst = torch.nan_to_num(ez.amax(1), nan=0.0, posinf=0.0)
    lse = out["lse"]
    lp = torch.where(torch.isfinite(lse)[:, None], z - lse[:, None], 0.0)
    p = torch.exp(lp)
    gap = torch.where(p > 0, p * (lp.abs() + out["entropy"].abs().nan_to_num()[:, None]), 0.0).sum(1)
    # sums of 32 logits in a lane and their joins lengthen the way by 64 additions
    more = 64 * U
    tol["lse"] = tol["lse"] + worst + more
    tol["logprob"] = tol["logprob"] + 2 * worst + more
    tol["entropy"] = tol["entropy"] + 2 * worst * (1 + gap.nan_to_num()) + more * (1 + gap.nan_to_num())
    return out, tol


def linear_logprobs_grad(hidden, weight, tokens, lse, ent, g, d, scale):
    """((dhidden, dweight), bounds without the last rounding), for lse (with its rest) and entropy as given."""
    t = hidden.dtype
    z, ez = logits(hidden, weight, scale)
    dz, e = so.token_logprobs_grad(z, tokens, lse, ent, g, d)
    none = (lse == -math.inf)[:, None]
    lp = torch.where(none, 0.0, z - lse.double()[:, None])
    p = torch.where(none, 0.0, torch.exp(lp))
    gg = g.double().abs()[:, None]
    dd = torch.zeros_like(gg) if d is None else d.double().abs()[:, None]
    hh = torch.zeros_like(gg) if ent is None else ent.double().abs()[:, None]
    flat = torch.where(p > 0, lp.abs(), 0.0)
    e = e + p * ez.exp() * ez * (gg + dd * (flat + hh + 1))
    sc = abs(float(torch.tensor(scale, dtype=torch.float32)))
    dz, e = dz * float(torch.tensor(scale, dtype=torch.float32)), e * sc
    # as operands, dz and the hidden states are bf16, two bf16 values, or three; either has a factor of the row taken out
    # or put in, an fp32 rounding or two each
    r = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -16, torch.float32: 2.0 ** -24}[t]
    e = e + (r + 4 * U) * (dz.abs() + e)
    parts = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}[t]
    h, w = hidden.double(), weight.double()
    eh = h.abs() * (r + 2 * U)
    dh, dw = dz @ w, dz.t() @ h
    e_dh = e @ w.abs() + terms(t, dz.shape[1], parts) * ((dz.abs() + e) @ w.abs()) + 4 * U * dh.abs()
    e_dw = e.t() @ (h.abs() + eh) + dz.abs().t() @ eh + terms(t, dz.shape[0], parts) * ((dz.abs() + e).t() @ (h.abs() + eh))
    return (dh, dw), (e_dh, e_dw)


# ------------------------------------------------- orthogonalised updates
USUAL = (3.4445, -4.7750, 2.0315)


def newton_schulz(x, steps, coefficients, eps, noise=None, dtype=torch.float32):
    """x (rows, cols) orthogonalised in 64 bits.  With a generator as `noise`, every rounding of the kernel is put in
    as a random error of the size of its bound: 2^-22 of what two fp16 parts keep (2^-11 of the operands of a bf16
    update's last products, which are the first parts alone), and of a product's sum 2 U of the root of the number
    of its terms (three for each k) times the root of the sum of their squares."""
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in coefficients)
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x

    def signs(v):
        return torch.randint(0, 2, v.shape, generator=noise, dtype=torch.float64).to(v.device) * 2 - 1

    def keep(v, bits=2.0 ** -22):
        return v if noise is None else v + signs(v) * (bits * v.abs() + 2.0 ** -37)

    def product(p, q, single):
        if noise is not None and single:
            # one rounding of a matrix, and of what is multiplied with it
            p, q = keep(p, 2.0 ** -11), keep(q, 2.0 ** -11)
        v = p @ q
        return v if noise is None else v + signs(v) * 2 * U * math.sqrt(3 * p.shape[1]) * ((p * p) @ (q * q)).sqrt()
    x = keep(x / (x.norm() + float(torch.tensor(eps, dtype=torch.float32))))
    for step in range(steps):
        single = dtype == torch.bfloat16 and step and step + 1 == steps and min(x.shape) >= 256
        gram = keep(product(x, x.t(), single))
        poly = keep(b * gram + c * product(gram, gram, single))
        x = keep(a * x + product(poly, x, single))
    return x.t() if tall else x
