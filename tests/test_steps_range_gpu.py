"""The training-step operators on the GPU at the ends of their ranges: far
logits, large means, long rows, other streams.  Bounds as in test_steps_gpu.
"""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
import step_oracle as so
from parity_util import say
from test_steps_gpu import BF16, DEV, F16, F32, gen

pytestmark = pytest.mark.gpu


# ---------------------------------------- logits between 2^24 and the type's end
def far_logits(value, rows, vocab, dtype):
    """Rows whose masked or whole logits lie at `value` (negative), among ordinary ones; some maxima at -value."""
    g = gen(vocab)
    z = torch.randn(8, vocab, generator=g, dtype=torch.float64) * 2
    z[0] = value                                         # nothing but masked ones
    z[1] = value
    z[1, vocab // 2] = 0.5                               # one left
    z[2, :vocab // 2] = value                            # whole lanes, waves and slices masked
    z[3] = value * (1 + torch.arange(vocab) % 3 * torch.finfo(dtype).eps * 2)
    z[4] = -math.inf
    z[4, ::2] = value
    z[5, vocab // 3] = -value                            # a far maximum
    z[6] = -value
    z[7, torch.rand(vocab, generator=g) < 0.7] = value
    return z.repeat(-(-rows // 8), 1)[:rows].to(dtype)


@pytest.mark.parametrize("rows,vocab,top", [(8, 300, 5), (1024, 300, 0), (1024, 777, 3), (8, 9001, 0), (8, 9001, 7), (8, 70001, 0),
                                            (8, 70000, 4)])
@pytest.mark.parametrize("zt,value", [(zt, v) for zt in (F32, BF16) for v in (-3e7, -1e9, -1e10, -1e12, -1e20, -1e30)]
                         + [(F16, -6e4), (F32, -2.0 ** 24), (F32, -2.0 ** 24 - 2), (F32, -2.0 ** 31), (F32, -3.4e38)])
def test_token_logprobs_of_far_logits(zt, value, rows, vocab, top):
    z = far_logits(value, rows, vocab, zt)
    tok = (torch.arange(rows) * 13 + vocab // 2) % vocab
    say("token_logprobs of far logits", zt, value, rows, vocab, top)
    zd, td = z.to(DEV), tok.to(DEV)
    p = rsx.token_logprobs(zd, td, top)
    ref, tol = so.token_logprobs(z, tok, top)
    for k, r in ref.items():
        got = getattr(p, k)
        if k == "top_token":
            assert torch.equal(got.cpu(), r), k
        else:
            so.close(got, r, tol[k] + 1.01 * so.rounding(r, F32), k)
    g, h = torch.randn(rows, generator=gen(1)), torch.full((rows,), 0.5)
    dz = rsx.token_logprobs_grad(zd, td, p.lse, g.to(DEV), p.entropy, h.to(DEV))
    rz, tz = so.token_logprobs_grad(z, tok, p.lse.cpu(), p.entropy.cpu(), g, h)
    so.close(dz, rz, tz + 1.01 * so.rounding(rz, zt), "dlogits")


@pytest.mark.parametrize("zt", [F32, BF16, F16])
@pytest.mark.parametrize("h", [-1e9, 1e20, -1e30, 3.4e38])
@pytest.mark.parametrize("vocab", [37, 9000])
def test_masked_logits_have_no_gradient_whatever_the_entropys(vocab, h, zt):
    z = torch.randn(6, vocab, generator=gen(vocab))
    z[:, 1::3] = torch.finfo(zt).min
    z[:, 2::3] = -math.inf
    z[:, 3::9] = -300.0                               # of no weight in 32 bits either
    z = z.to(zt)
    tok = torch.tensor([0, 1, 2, 3, 4, -1])
    say("masked logits, dentropy", h, zt, vocab)
    zd, td = z.to(DEV), tok.to(DEV)
    p = rsx.token_logprobs(zd, td)
    g, hs = torch.randn(6, generator=gen(2)), torch.full((6,), h)
    dz = rsx.token_logprobs_grad(zd, td, p.lse, g.to(DEV), p.entropy, hs.to(DEV))
    rz, tz = so.token_logprobs_grad(z, tok, p.lse.cpu(), p.entropy.cpu(), g, hs)
    masked = z.float() <= -300
    got = dz.cpu()
    assert (got[masked & (torch.arange(vocab) != tok[:, None])] == 0).all()
    own = masked.gather(1, tok.clamp(min=0)[:, None])[:, 0] & (tok >= 0)   # a masked token has its own gradient alone
    assert torch.equal(got.gather(1, tok.clamp(min=0)[:, None])[:, 0][own], g.to(zt)[own])
    if abs(h) < 1e38 and zt != F16:                   # else what is not masked leaves the type
        so.close(dz, rz, tz + 1.01 * so.rounding(rz, zt), "dlogits")


def log_probabilities(z):
    """Of all tokens of rows without NaNs, in 64 bits, and a bound of their error that counts no rounding of z or lse."""
    z = z.double()
    c = z - z.amax(1, keepdim=True)
    p = torch.exp(c)
    s = p.sum(1, keepdim=True)
    gap = torch.where(p > 0, p * -c, 0.0).sum(1, keepdim=True) / s
    # as step_oracle.token_logprobs: the sum's relative error, then a difference and a logarithm
    return c - torch.log(s), so.U * (z.shape[1] / 256 + 128 + 4 + 4 * gap) + 4 * so.U * (c.abs() + torch.log(s))


@pytest.mark.parametrize("level", [0.0, -16384.0, 2.0 ** 20, 2.0 ** 22, -2.0 ** 22, 2.0 ** 24 - 40])
@pytest.mark.parametrize("rows,vocab,zt", [(6, 2000, F32), (1030, 4000, F32), (5, 30001, F32), (3, 200001, F32), (300, 50000, F32),
                                           (3, 70001, BF16)])
def test_rising_rows_far_from_zero(rows, vocab, zt, level):
    """The maximum rises in most steps: what was summed before it has to follow."""
    z = torch.linspace(0, 8, vocab, dtype=torch.float64) + torch.randn(rows, vocab, generator=gen(vocab)) * 0.5 + level
    z = z.to(zt)
    tok = torch.arange(rows) * 7 % vocab
    say("rising rows", rows, vocab, zt, level)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV))
    lp, tol = log_probabilities(z)
    want, tol = lp.gather(1, tok[:, None])[:, 0], tol.gather(1, tok[:, None])[:, 0]
    so.close(p.logprob, want, tol + 1.01 * so.rounding(want, F32), "logprob")
    ref, rtol = so.token_logprobs(z, tok, 0)
    so.close(p.entropy, ref["entropy"], rtol["entropy"] + 1.01 * so.rounding(ref["entropy"], F32), "entropy")
    so.close(p.lse, ref["lse"], rtol["lse"] + 1.01 * so.rounding(ref["lse"], F32), "lse")


def level_logits(rows, vocab, level, dtype):
    """Logits around `level`, and tokens that are the most likely, a likely or any other one."""
    g = gen(vocab + rows)
    z = (torch.randn(rows, vocab, generator=g) * 2 + level).to(dtype)
    best = torch.argsort(z.float(), dim=1, descending=True, stable=True)
    tok = best.gather(1, torch.tensor([0, min(2, vocab - 1), vocab // 2]).repeat(rows)[:rows, None])[:, 0]
    return z, tok


@pytest.mark.parametrize("level", [0.0, 900.0, -16384.0, 16384.0, 2.0 ** 22])
@pytest.mark.parametrize("rows,vocab,top,zt", [(6, 40, 8, F32), (1030, 1000, 5, F32), (5, 9001, 16, F32), (3, 70001, 64, F32),
                                               (5, 9001, 8, BF16), (3, 131072, 8, BF16)])
def test_alternatives_have_the_digits_of_the_log_probabilities(rows, vocab, top, zt, level):
    z, tok = level_logits(rows, vocab, level, zt)
    say("alternatives at a level", rows, vocab, top, zt, level)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV), top)
    lp, tol = log_probabilities(z)
    at = p.top_token.cpu().long()
    want = lp.gather(1, at)
    so.close(p.top_logprob, want, tol.gather(1, at) + 1.01 * so.rounding(want, F32), "top_logprob")
    # one token, one value
    mine = p.top_token == tok.to(DEV)[:, None]
    row = mine.any(1)
    assert row.any()
    assert torch.equal(p.top_logprob[mine], p.logprob[row])


@pytest.mark.parametrize("level", [0.0, 900.0, -16384.0, 16384.0, 2.0 ** 22])
@pytest.mark.parametrize("rows,vocab,zt", [(6, 40, F32), (1030, 1000, F32), (5, 9001, F32), (3, 70001, F32), (5, 9001, BF16)])
def test_gradient_has_the_digits_of_the_log_probabilities(rows, vocab, zt, level):
    """Against the logits alone: no rounding of lse's size counts."""
    z, tok = level_logits(rows, vocab, level, zt)
    g, h = torch.randn(rows, generator=gen(1)), torch.randn(rows, generator=gen(2))
    say("gradient at a level", rows, vocab, zt, level)
    zd, td = z.to(DEV), tok.to(DEV)
    p = rsx.token_logprobs(zd, td)
    lp, tol = log_probabilities(z)
    ent = -(lp.exp() * lp).sum(1)
    whole, e_lse = z.double().amax(1) - lp.amax(1), tol.amin(1)
    two = p.lse.cpu().double() + p.lse_rest.cpu().double()
    assert ((two - whole).abs() <= e_lse + 2 * so.U ** 2 * whole.abs() + 2.0 ** -52 * whole.abs()).all()
    dz = rsx.token_logprobs_grad(zd, td, p.lse, g.to(DEV), p.entropy, h.to(DEV), lse_rest=p.lse_rest)
    e_ent = so.token_logprobs(z, tok, 0)[1]["entropy"][:, None] + so.rounding(ent, F32)[:, None]
    prob, g, h, ent = lp.exp(), g.double()[:, None], h.double()[:, None], ent[:, None]
    hit = torch.zeros_like(lp).scatter_(1, tok[:, None], 1.0)
    want = g * hit - prob * (g + h * (lp + ent))
    # p's relative error is lp's; lp and the entropy again as factors of h; then the products' roundings
    size = prob * (g.abs() + h.abs() * (lp.abs() + ent))
    e = size * (tol + so.U * (12 + 4 * lp.abs())) + prob * h.abs() * (tol + e_ent) + 2 * so.U * g.abs() * hit + 2.0 ** -120
    so.close(dz, want, e + 1.01 * so.rounding(want, zt), "dlogits")


@pytest.mark.parametrize("vocab", [64, 9000])
@pytest.mark.parametrize("zt,value", [(F32, -3.4e38), (F32, -1e10), (F32, 1e30), (BF16, -1e9), (BF16, torch.finfo(BF16).min),
                                      (F16, torch.finfo(F16).min)])
def test_rows_of_one_far_value_are_uniform(zt, value, vocab):
    """The softmax of equal logits is 1 / vocab, and so is its gradient, also where lse itself is the value."""
    z = torch.full((3, vocab), value).to(zt)
    z[1, 1::2] = -math.inf
    tok = torch.tensor([0, 2, -1])
    say("rows of one far value", zt, value, vocab)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV))
    g, h = torch.tensor([1.0, -0.5, 2.0]), torch.tensor([0.0, 0.3, 0.7])
    dz = rsx.token_logprobs_grad(z.to(DEV), tok.to(DEV), p.lse, g.to(DEV), p.entropy, h.to(DEV), lse_rest=p.lse_rest)
    n = torch.tensor([vocab, vocab // 2, vocab], dtype=torch.float64)[:, None]
    there = (z != -math.inf).double()
    ok = (tok >= 0).double()[:, None]
    hit = torch.zeros(3, vocab, dtype=torch.float64).scatter_(1, tok.clamp(min=0)[:, None], 1.0) * ok
    want = g.double()[:, None] * (hit - there / n * ok)  # all alike: the entropy is at its largest and has no slope
    # ln n has two roundings, p one exponential; log p + H leaves those of ln n, each of a size of at most ln 9000
    e = there / n * so.U * 16 * (3 + 10) + 2 * so.U * hit
    so.close(dz, want, e + 1.01 * so.rounding(want, zt), "dlogits")
    assert torch.equal(p.entropy.cpu() > 0, torch.ones(3, dtype=torch.bool))


# --------------------------------------------------- rows around a large mean
def layer_norm_bounds(x, w, b, eps):
    """((y, mean, rstd), their bounds) in which the mean's size counts in its own last rounding and in products with U^2 alone."""
    x = x.double()
    d = x.shape[1]
    n = d / 64 + 64                                          # additions one after another
    eps = float(torch.tensor(eps, dtype=F32))
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(d, dtype=torch.float64) if b is None else b.double()
    y = c * rstd * w + b
    e0 = (n + 3) * so.U * x.abs().mean(1, keepdim=True)      # a mean from one sum is off by that
    e_mean = (n + 4) * so.U * (c.abs().mean(1, keepdim=True) + e0)       # the mean of the differences from it
    e_c = e_mean + 3 * so.U * (c.abs() + e0)
    e_var = (n + 6) * so.U * (var + e0.square()) + 2 * e0 * e_mean + e_mean.square()
    most, least = ((var - e_var).clamp(min=0) + eps).rsqrt(), (var + e_var + eps).rsqrt()
    e_rstd = torch.maximum(most - rstd, rstd - least) + 4 * so.U * most
    e_y = w.abs() * (c.abs() * e_rstd + e_c * (rstd + e_rstd)) + 3 * so.U * ((w * c * rstd).abs() + b.abs())
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0], e_rstd[:, 0])


@pytest.mark.parametrize("rows,dim", [(5, 2), (9, 26), (9, 30), (6, 61), (4200, 117), (7, 300), (5, 1000), (6, 2047), (4097, 3001),
                                      (3, 6000), (3, 11000), (2, 16385), (2, 40001)])
@pytest.mark.parametrize("xt,level,spread", [(F32, 1e4, 0.0), (F32, 1e4, 0.01), (F32, -3e6, 2.0), (F32, 0.1, 0.0), (F32, 1e17, 1e16), (F32, 1e20, 1e19),
                                             (F16, 6e4, 0.0), (F16, 1000.0, 1.0), (BF16, 59904.0, 0.0), (BF16, -256.0, 2.0)])
def test_layer_norm_around_a_large_mean(xt, level, spread, rows, dim):
    g = gen(dim)
    few = min(rows, 9)  # more rows repeat these
    x = (level + torch.randn(few, dim, generator=g, dtype=torch.float64) * spread).to(xt)
    w, b = (torch.randn(dim, generator=g) * 0.3 + 1).to(xt), (torch.randn(dim, generator=g) * 0.3).to(xt)
    say("layer_norm around a mean", xt, level, spread, rows, dim)
    y, mean, rstd = rsx.layer_norm(x.repeat(-(-rows // few), 1)[:rows].contiguous().to(DEV), w.to(DEV), b.to(DEV))
    (ry, rm, rr), (ty, tm, tr) = layer_norm_bounds(x, w, b, 1e-5)
    for at in (0, rows - few):
        part = slice(at, at + few)
        back = torch.arange(at, at + few) % few
        so.close(mean[part], rm[back], (tm + 1.01 * so.rounding(rm, F32))[back], "mean")
        so.close(rstd[part], rr[back], (tr + 1.01 * so.rounding(rr, F32))[back], "rstd")
        so.close(y[part], ry[back], (ty + 1.01 * so.rounding(ry, xt))[back], "y")


@pytest.mark.parametrize("rows,dim", [(4, 3), (4, 40), (4099, 200), (4, 3000), (4, 9000), (3, 33000)])
def test_layer_norm_statistics_of_rows_without_a_mean(rows, dim):
    x = torch.randn(rows, dim, generator=gen(dim))
    x[0, dim // 2], x[1, 0], x[2, dim - 1] = math.inf, math.nan, -math.inf
    say("layer_norm with infinities", rows, dim)
    y, mean, rstd = rsx.layer_norm(x.to(DEV))
    assert torch.isnan(y[:3]).all() and torch.isnan(rstd[:3]).all()
    assert mean[:3].tolist()[::2] == [math.inf, -math.inf] and math.isnan(mean[1].item())
    (ry, rm, rr), (ty, tm, tr) = layer_norm_bounds(x[3:], None, None, 1e-5)
    if rows > 3:
        so.close(y[3:], ry, ty + 1.01 * so.rounding(ry, F32), "y")
        so.close(rstd[3:], rr, tr + 1.01 * so.rounding(rr, F32), "rstd")


# ------------------------------------------------------- another stream's memory
@pytest.mark.parametrize("given", ["object", "handle"])
def test_functions_on_a_stream_take_no_memory_from_the_current_one(given):
    """A block just freed on the current stream may still be written there; a call on another one must not be given it."""
    rows, dim = 3000, 1000
    g = gen(6)
    x, dy = torch.randn(rows, dim, generator=g).to(DEV), torch.randn(rows, dim, generator=g).to(DEV)
    tok = torch.randint(0, dim, (rows,), generator=g).to(DEV)
    want = rsx.layer_norm(x)
    back = rsx.layer_norm_grad(dy, x, *want[1:])
    lp = rsx.token_logprobs(x, tok, 3)
    dz = rsx.token_logprobs_grad(x, tok, lp.lse, lp.logprob, lse_rest=lp.lse_rest)
    rows_of = rsx.embedding(x, tok)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    arg = s if given == "object" else s.cuda_stream
    torch.cuda.synchronize()
    freed = [torch.empty(rows, dim, device=DEV) for _ in range(3)]
    taken = {t.data_ptr() for t in freed}
    del freed
    got = rsx.layer_norm(x, stream=arg)
    b = rsx.layer_norm_grad(dy, x, *got[1:], stream=arg)
    l2 = rsx.token_logprobs(x, tok, 3, stream=arg)
    d2 = rsx.token_logprobs_grad(x, tok, l2.lse, l2.logprob, stream=arg, lse_rest=l2.lse_rest)
    r2 = rsx.embedding(x, tok, stream=arg)
    assert not taken & {t.data_ptr() for t in (got[0], b[0], d2, r2)}
    torch.cuda.current_stream().wait_stream(s)
    for a, c in zip((*want, *back, lp.logprob, lp.top_token, dz, rows_of), (*got, *b, l2.logprob, l2.top_token, d2, r2)):
        assert torch.equal(a, c)
    # handle 0 is the default stream, from any other
    with torch.cuda.stream(s):
        y = rsx.layer_norm(x, stream=0)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


# ------------------------------------------------------- rows of 2^25 and more elements
def test_layer_norm_gradient_of_a_row_beyond_2_27_elements():
    """The launches' work-items pass 32 bits."""
    dim = 2 ** 27 + 5
    g = torch.Generator(device=DEV).manual_seed(3)
    x, dy = torch.randn(1, dim, generator=g, device=DEV).bfloat16(), torch.randn(1, dim, generator=g, device=DEV).bfloat16()
    say("layer_norm_grad of", dim)
    dx, dw, db = rsx.layer_norm_grad(dy, x, torch.full((1,), 0.5, device=DEV), torch.full((1,), 2.0, device=DEV))
    assert torch.equal(db, dy[0])                            # a sum of one; zeros of either sign are equal
    xhat = (x[0].float() - 0.5) * 2
    assert torch.equal(dw, (dy[0].float() * xhat).bfloat16())
    c1, c2 = dy[0].double().mean(), (dy[0].double() * xhat.double()).mean()
    want = 2 * (dy[0].float() - c1.float() - xhat * c2.float())
    # additions one after another: the row's share of a lane, and the lanes; means of terms of about 1 and 4
    tol = (dim / 2 ** 13 + 80) * so.U * 2 * (1 + 4 * xhat.abs()) + 8 * so.U * (1 + dy[0].float().abs() + xhat.abs())
    assert ((dx[0].float() - want).abs() <= tol + 1.01 * so.rounding(want, BF16)).all()


@pytest.mark.skipif(not torch.cuda.is_available() or torch.cuda.mem_get_info()[1] < 240 << 30, reason="needs 205 GiB")
def test_layer_norm_gradient_of_many_rows_of_2_25_elements():
    """512 rows, expanded: the columns' pass has more work-items than 32 bits count."""
    rows, dim = 512, 2 ** 25 + 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 205 << 30:
        pytest.skip("needs 205 GiB free")
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dy = torch.randn(1, dim, generator=g, device=DEV), torch.randn(1, dim, generator=g, device=DEV)
    rstd = torch.linspace(0.5, 1.5, rows, device=DEV)
    say("layer_norm_grad of", rows, dim)
    dx, dw, db = rsx.layer_norm_grad(dy.expand(rows, dim), x.expand(rows, dim), torch.zeros(rows, device=DEV), rstd)
    total = rstd.double().sum()
    for a in range(0, dim, 1 << 22):                         # in pieces: 64 bits
        part = slice(a, min(a + (1 << 22), dim))
        d, v = dy[0, part].double(), x[0, part].double()
        assert ((dw[part] - d * v * total).abs() <= (rows + 8) * so.U * (d * v).abs() * total).all()
        assert ((db[part] - d * rows).abs() <= (rows + 4) * so.U * d.abs() * rows).all()
    c1, c2 = dy.double().mean(), (dy.double() * x.double()).mean()
    for r in (0, 1, 255, rows - 1):
        k = rstd[r].double()
        for a in (0, dim // 2, dim - (1 << 20)):
            d, v = dy[0, a:a + (1 << 20)].double(), x[0, a:a + (1 << 20)].double() * k
            want = k * (d - c1 - v * c2 * k)
            tol = (dim / 2 ** 12 + 80) * so.U * k * (1 + 2 * v.abs()) + 8 * so.U * (1 + d.abs() + v.abs())
            assert ((dx[r, a:a + (1 << 20)] - want).abs() <= tol + so.rounding(want, F32)).all()
    del dx, dw, db
    torch.cuda.empty_cache()


def test_layer_norm_of_rows_without_elements():
    """The mean of nothing is no number, and not what the memory held."""
    for _ in range(3):
        held = [torch.zeros(1000, device=DEV) for _ in range(4)]
        del held
        y, mean, rstd = rsx.layer_norm(torch.empty(1000, 0, device=DEV))
        assert y.shape == (1000, 0) and torch.isnan(mean).all() and torch.isnan(rstd).all()
    dx, dw, db = rsx.layer_norm_grad(y, y, mean, rstd)
    assert dx.shape == (1000, 0) and dw.numel() == 0 and db.numel() == 0


@pytest.mark.parametrize("rows,dim", [(5, 3), (5, 40), (4099, 200), (5, 700), (5, 3000), (4, 9000), (3, 33000)])
@pytest.mark.parametrize("kind", ["signs", "level", "uniform", "one"])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_layer_norm_of_rows_whose_sums_leave_32_bits(xt, kind, rows, dim):
    """Finite values, with a finite mean and differences that fp32 does not all hold."""
    few, g = min(rows, 5), gen(dim)
    x = {"signs": lambda: torch.where(torch.arange(dim) % 2 == 0, 3e38, -2e38).expand(few, dim).double(),
         "level": lambda: 1e38 + 1e37 * torch.randn(few, dim, generator=g, dtype=torch.float64),
         "uniform": lambda: 3e38 * torch.rand(few, dim, generator=g, dtype=torch.float64),
         "one": lambda: torch.cat([torch.full((few, 1), -3.3e38), torch.full((few, dim - 1), 3.3e38)], 1).double()}[kind]().to(xt)
    w, b = (torch.randn(dim, generator=g) * 0.3 + 1).to(xt), (torch.randn(dim, generator=g) * 0.3).to(xt)
    say("layer_norm of sums past fp32", xt, kind, rows, dim)
    xd = x.repeat(-(-rows // few), 1)[:rows].contiguous().to(DEV)
    ck = rsx.Checkpoint(xd.shape, DEV)
    y, mean, rstd = rsx.layer_norm(xd, w.to(DEV), b.to(DEV), checkpoint=ck)
    (ry, rm, rr), (ty, tm, tr) = layer_norm_bounds(x, w, b, 1e-5)
    so.close(mean[:few], rm, tm + 1.01 * so.rounding(rm, F32), "mean")
    so.close(rstd[:few], rr, tr + 1.01 * so.rounding(rr, F32), "rstd")
    so.close(y[:few], ry, ty + 1.01 * so.rounding(ry, xt), "y")
    codes, scales = so.checkpoint(x)
    assert torch.equal(ck.codes[:few].cpu(), codes) and torch.equal(ck.scales[:few].cpu(), scales)
