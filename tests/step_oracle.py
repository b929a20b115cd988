"""The training-step operators from their definitions, in 64 bits on the CPU,
with bounds on what a kernel that holds its sums in fp32 may differ by.

U is half a step of fp32, the error of one rounding.  A sum of n terms in any
order is off by at most n * U times the sum of the terms' magnitudes.
"""
import math

import torch

U = 2.0 ** -24
BLOCK = 32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(ref, dtype):
    """One rounding of `ref` to `dtype`, subnormals included."""
    f = torch.finfo(dtype)
    return half(dtype) * ref.abs() + f.smallest_normal * f.eps


def close(got, ref, tol, what=""):
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    over = ((got - ref).abs() - tol.expand_as(ref).double())[fine]
    if over.numel():
        worst = over.max().item()
        assert worst <= 0, f"{what}: {worst} over the bound, {(over > 0).sum().item()} of {over.numel()} values"


# -------------------------------------------------------------- embedding
def embedding(table, tokens, scale, first):
    t = tokens.reshape(-1).long() - first
    ok = (t >= 0) & (t < table.shape[0])
    out = torch.zeros(t.numel(), table.shape[1], dtype=torch.float64)
    out[ok] = table[t[ok]].double() * float(torch.tensor(scale, dtype=torch.float32))
    return out


def embedding_grad(dout, tokens, vocab, scale, first, old=None):
    """(gradient, bound without the last rounding)."""
    d = dout.reshape(-1, dout.shape[-1]).double()
    t = tokens.reshape(-1).long() - first
    ok = (t >= 0) & (t < vocab)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    total = torch.zeros(vocab, d.shape[1], dtype=torch.float64)
    size = torch.zeros_like(total)
    count = torch.zeros(vocab, 1, dtype=torch.float64)
    total.index_add_(0, t[ok], d[ok])
    size.index_add_(0, t[ok], d[ok].abs())
    count.index_add_(0, t[ok], torch.ones(int(ok.sum()), 1, dtype=torch.float64))
    grad = total * scale
    tol = (count + 2) * U * size * abs(scale)
    if old is not None:
        grad = grad + old.double()
        tol = tol + 2 * U * (grad.abs() + old.double().abs())
    return grad, tol


# -------------------------------------------------------------- layer norm
def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) and their bounds without the last rounding; x (rows, dim)."""
    x = x.double()
    d = x.shape[1]
    n = d / 64 + 64  # additions one after another, in a lane and across lanes
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    rstd = (var + eps).rsqrt()
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(d, dtype=torch.float64) if bias is None else bias.double()
    y = c * rstd * w + b
    e_mean = (n + 2) * U * x.abs().mean(1, keepdim=True)
    # the variance: its sum, and the mean's error (squared: the differences sum to 0 around the mean)
    r_rstd = 0.5 * ((n + 6) * U + e_mean.square() * rstd.square()) + 4 * U
    xhat = c * rstd
    t_y = w.abs() * (xhat.abs() * (r_rstd + 4 * U) + e_mean * rstd) + 2 * U * ((w * xhat).abs() + b.abs())
    return (y, mean[:, 0], rstd[:, 0]), (t_y, e_mean[:, 0], (rstd * r_rstd)[:, 0])


def layer_norm_grad(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) and their bounds without the last rounding; mean and rstd as given."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    r, d = x.shape
    n = d / 64 + 64
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    xhat = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xhat * c2)
    e1 = (n + 4) * U * g.abs().mean(1, keepdim=True)
    e2 = (n + 8) * U * (g * xhat).abs().mean(1, keepdim=True)
    t_dx = rstd.abs() * (e1 + xhat.abs() * e2 + 6 * U * (g.abs() + c1.abs() + (xhat * c2).abs()))
    t_dw = (r + 6) * U * (dy * xhat).abs().sum(0)
    t_db = (r + 2) * U * dy.abs().sum(0)
    return (dx, (dy * xhat).sum(0), dy.sum(0)), (t_dx, t_dw, t_db)


# ------------------------------------------------------------- checkpoints
def checkpoint(x):
    """(codes, scale bytes) of x (rows, dim)."""
    x = x.double()
    r, d = x.shape
    nb = -(-d // BLOCK)
    pad = torch.zeros(r, nb * BLOCK, dtype=torch.float64)
    pad[:, :d] = x
    b = pad.view(r, nb, BLOCK)
    most = b.abs().amax(2)  # NaN where a NaN is
    bad = ~torch.isfinite(most)
    e = torch.frexp(torch.where(bad, 0.0, most))[1] - 1  # 2^e <= most < 2^(e+1)
    byte = torch.where(most > 0, (e - 6 + 127).clamp(min=0), 0)
    step = torch.ldexp(torch.ones_like(most), byte - 127)
    q = torch.round(b / step[:, :, None]).clamp(-127, 127)
    q = torch.where(bad[:, :, None], 0.0, q)
    return q.view(r, -1)[:, :d].to(torch.int8), torch.where(bad, 255, byte).to(torch.uint8)


def checkpoint_values(codes, scales):
    codes, scales = codes.cpu(), scales.cpu()
    step = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64), scales.int() - 127)
    step = torch.where(scales == 255, math.nan, step)
    return codes.double() * step.repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]


# ---------------------------------------------------- token log probabilities
def token_logprobs(z, tokens, top):
    """A dict of results and one of bounds; z (rows, vocab)."""
    z = z.double()
    r, v = z.shape
    n = v / 256 + 128
    bad = (torch.isnan(z) | (z == math.inf)).any(1)
    none = (z == -math.inf).all(1)
    m = torch.where(none | bad, 0.0, torch.where(torch.isnan(z), -math.inf, z).amax(1))
    c = z - m[:, None]
    p = torch.exp(c)
    s = p.sum(1)
    gap = torch.where(p > 0, p * -c, 0.0).sum(1) / torch.where(none, 1.0, s)
    ln_s = torch.log(s)
    lse = torch.where(bad, math.nan, m + ln_s)
    ok = (tokens >= 0) & (tokens < v)
    zt = z.gather(1, tokens.long().clamp(0, v - 1)[:, None])[:, 0]
    lp = torch.where(none, -math.inf, zt - m - ln_s)
    lp = torch.where(bad, math.nan, lp)
    lp = torch.where(ok, lp, 0.0)
    ent = torch.where(bad, math.nan, torch.where(none, 0.0, ln_s + gap))
    # relative error of s: its sum, one exponential each, and the exponents' roundings
    r_s = U * (n + 4 + 4 * gap)
    safe = lambda t: torch.where(torch.isfinite(t), t, 0.0)  # noqa: E731
    gap2 = torch.where(p > 0, p * c * c, 0.0).sum(1) / torch.where(none, 1.0, s)
    tol = {"lse": safe(r_s + 4 * U * (ln_s.abs() + lse.abs())),
           "logprob": safe(r_s + 4 * U * ((zt - m).abs() + ln_s.abs())),
           "entropy": safe(2 * r_s * (1 + gap) + 4 * U * (ln_s.abs() + gap + gap2))}
    out = {"lse": lse, "logprob": lp, "entropy": ent}
    if top:
        key = torch.where(torch.isnan(z), -math.inf, z)
        # stable by index within equal values; a NaN below -inf
        order = torch.argsort(torch.isnan(z).long(), dim=1, stable=True)
        order = order.gather(1, torch.argsort(key.gather(1, order), dim=1, descending=True, stable=True))
        best = order[:, :top]
        out["top_token"] = best.int()
        zb = z.gather(1, best)
        out["top_logprob"] = torch.where(none[:, None], -math.inf, torch.where(bad[:, None], math.nan, zb - lse[:, None]))
        tol["top_logprob"] = safe(r_s + 4 * U * (ln_s.abs() + lse.abs()))[:, None] + 2 * U * safe(zb.abs())
    # results are fp32: what is past its range is an infinity there
    most = torch.finfo(torch.float32).max
    out = {k: torch.where(r.abs() > most, torch.sign(r) * math.inf, r) if r.is_floating_point() else r for k, r in out.items()}
    return out, tol


def token_logprobs_grad(z, tokens, lse, ent, g, h):
    """(dlogits, bound without the last rounding) for lse and ent as given."""
    z, lse = z.double(), lse.double()[:, None]
    v = z.shape[1]
    none = lse == -math.inf
    lp = z - torch.where(none, 0.0, lse)
    p = torch.exp(lp)
    ok = (tokens >= 0) & (tokens < v)
    g = torch.where(ok, g.double(), 0.0)[:, None]
    h = torch.zeros_like(g) if h is None else h.double()[:, None]
    ent = torch.zeros_like(g) if ent is None else ent.double()[:, None]
    flat = torch.where(p > 0, lp, 0.0)
    dz = -p * (g + h * (flat + ent))
    hit = torch.zeros_like(z).scatter_(1, tokens.long().clamp(0, v - 1)[:, None], 1.0) * ok[:, None]
    dz = torch.where(none, 0.0, dz + g * hit)
    size = p * (g.abs() + h.abs() * (flat.abs() + ent.abs()))
    tol = size * U * (12 + 4 * flat.abs()) + 2 * U * g.abs() * hit + 2.0 ** -120
    return dz, torch.where(none | torch.isnan(tol), 0.0, tol)
