"""The step's matrix products on the GPU against their definitions in 64 bits.

Bounds come from product_oracle: they count the fp32 roundings of a sum and the
roundings of operands, plus the one rounding to the output's type.  Inputs of
small whole numbers have results that every type holds exactly, and have to be
equal.
"""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
import product_oracle as po
import step_oracle as so
from parity_util import say
from test_steps_gpu import BF16, DEV, F16, F32, gen, rand, same_bits, untouched, wide_rows

pytestmark = pytest.mark.gpu


def place(host, pad):
    """`host` on the GPU, in a wider matrix with NaN on either side for pad > 0."""
    return wide_rows(host, pad) if pad else (None, host.to(DEV))


def fits(got, ref, tol, dtype, what):
    so.close(got.double(), ref, tol + 1.01 * so.rounding(ref, dtype), what)


# ------------------------------------------------------------ feed-forward
FFN = [  # rows, dim, hidden, type, activation, pad, kept
    (1, 1, 1, F32, "silu", 0, True), (1, 8, 8, BF16, "silu", 0, True), (1, 4096, 300, BF16, "gelu", 0, False),
    (2, 7, 3, F16, "relu", 1, True), (8, 520, 136, BF16, "silu", 0, True), (16, 257, 65, F32, "gelu_tanh", 3, True),
    (17, 96, 40, F16, "gelu", 0, True), (33, 1000, 17, BF16, "silu", 8, True), (64, 64, 64, F32, "relu", 0, True),
    (64, 65, 33, BF16, "gelu_tanh", 1, True), (65, 64, 64, BF16, "silu", 0, True), (65, 72, 136, F16, "gelu", 8, True),
    (100, 33, 47, F32, "silu", 0, True), (128, 128, 128, BF16, "relu", 0, True), (129, 264, 200, BF16, "gelu_tanh", 1, True),
    (200, 1, 300, BF16, "silu", 0, True), (300, 300, 1, F32, "gelu", 0, True), (257, 71, 129, F16, "silu", 3, True),
    (130, 1025, 513, F32, "gelu_tanh", 1, True), (1000, 136, 520, BF16, "silu", 0, True), (70, 8, 2000, BF16, "gelu", 0, True),
    (4, 200, 9001, BF16, "silu", 0, True), (33, 24, 5000, F32, "gelu", 0, True), (64, 5, 2048, F16, "relu", 1, True),
]


def block(g, rows, dim, hidden, t):
    x = rand(g, rows, dim, dtype=t)
    wg, wu = (rand(g, hidden, dim, dtype=t, scale=dim ** -0.5) for _ in range(2))
    return x, wg, wu, rand(g, dim, hidden, dtype=t, scale=hidden ** -0.5)


@pytest.mark.parametrize("rows,dim,hidden,t,act,pad,keep", FFN)
def test_feed_forward(rows, dim, hidden, t, act, pad, keep):
    say("feed_forward", rows, dim, hidden, t, act, pad)
    g = gen(rows + dim + hidden)
    host = block(g, rows, dim, hidden, t)
    x, wg, wu, wd = (place(h, pad)[1] for h in host)
    big, out = wide_rows(torch.zeros(rows, dim, dtype=t), pad)
    plan = rsx.FeedForward(x, wg, wu, wd, out, activation=act, keep=keep)
    plan()
    ref, tol = po.feed_forward(*host, act)
    fits(out, ref[0], tol[0], t, "out")
    assert pad == 0 or untouched(big, pad, dim)
    once = out.clone()
    plan()
    assert same_bits(once, out)
    if not keep:
        return
    fits(plan.gate, ref[1], tol[1], F32, "gate")
    fits(plan.up, ref[2], tol[2], F32, "up")
    dy = rand(g, rows, dim, dtype=t)
    wtype = F32 if rows % 2 else t
    dx_big, dx = wide_rows(torch.zeros(rows, dim, dtype=t), pad)
    old = [rand(g, hidden, dim, dtype=wtype), rand(g, hidden, dim, dtype=wtype), rand(g, dim, hidden, dtype=wtype)]
    placed = [wide_rows(o, pad) for o in old]
    for acc in (False, True):
        for (_, view), o in zip(placed, old):
            view.copy_(o)
        rsx.feed_forward_grad(place(dy, pad)[1], x, wg, wu, wd, plan.gate, plan.up, dx, *(v for _, v in placed), activation=act,
                              accumulate=acc)
        refs, tols = po.feed_forward_grad(dy, *host, plan.gate.cpu(), plan.up.cpu(), act)
        fits(dx, refs[0], tols[0], t, "dx")
        for what, (b, v), o, r, e in zip(("dw_gate", "dw_up", "dw_down"), placed, old, refs[1:], tols[1:]):
            if acc:
                r = r + o.double()
                e = e + 4 * so.U * (r.abs() + o.double().abs())
            fits(v, r, e, wtype, what)
            assert pad == 0 or untouched(b, pad, v.shape[1]), what
    assert pad == 0 or untouched(dx_big, pad, dim)


def whole(g, rows, cols, each, values=(-1, 1)):
    """Rows of zeros but for `each` whole numbers at random places."""
    m = torch.zeros(rows, cols)
    at = torch.randint(0, cols, (rows, each), generator=g)
    v = torch.tensor(values, dtype=torch.float32)[torch.randint(0, len(values), (rows, each), generator=g)]
    return m.scatter_(1, at, v)


EXACT = [  # rows, dim, hidden: of large tiles, middle ones, cut sums, few rows
    (2100, 520, 4200), (2048, 256, 8192), (700, 2056, 1000), (130, 4096, 264), (37, 3000, 1500), (5, 11008, 4099), (7, 136, 20000),
]


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("rows,dim,hidden", EXACT)
def test_feed_forward_whole_numbers(rows, dim, hidden, t):
    say("feed_forward whole", rows, dim, hidden, t)
    g = gen(rows)
    x, wg, wu, dy = whole(g, rows, dim, 3), whole(g, hidden, dim, dim // 4), whole(g, hidden, dim, dim // 4), whole(g, rows, dim, 3)
    wd = whole(g, dim, hidden, 4)  # of 7 x 136 x 20000 and the like the second product's k is cut
    dev = [m.to(DEV, t) for m in (x, wg, wu, wd, dy)]
    p = rsx.feed_forward(*dev[:4], activation="relu", keep=True)
    x, wg, wu, wd, dy = (m.double() for m in dev)
    gate, up = x @ wg.t(), x @ wu.t()  # at most 3
    s = gate.clamp(min=0) * up         # at most 9
    assert torch.equal(p.gate.double(), gate) and torch.equal(p.up.double(), up)
    assert torch.equal(p.out.double(), s @ wd.t())
    ds = dy @ wd
    dg, du = ds * up * (gate > 0), ds * gate.clamp(min=0)
    grads = rsx.feed_forward_grad(dev[4], *dev[:4], p.gate, p.up, dw_gate=torch.empty(hidden, dim, device=DEV),
                                  dw_up=torch.empty(hidden, dim, device=DEV), dw_down=torch.empty(dim, hidden, device=DEV),
                                  activation="relu")
    dx = dg @ wg + du @ wu
    assert torch.equal(grads[0], dx.to(t))
    for got, want in zip(grads[1:], (dg.t() @ x, du.t() @ x, dy.t() @ s)):
        assert torch.equal(got.double(), want)


def test_feed_forward_of_nothing():
    w, d = torch.randn(24, 16, device=DEV), torch.randn(16, 24, device=DEV)
    p = rsx.feed_forward(torch.empty(0, 16, device=DEV), w, w, d, keep=True)
    assert p.out.shape == (0, 16) and p.gate.shape == (0, 24)
    old = torch.ones_like(w), torch.ones_like(w), torch.ones_like(d)
    rsx.feed_forward_grad(p.out, p.out, w, w, d, p.gate, p.up, None, *old, accumulate=True)
    assert all((o == 1).all() for o in old)
    grads = rsx.feed_forward_grad(p.out, p.out, w, w, d, p.gate, p.up)
    assert all((o == 0).all() for o in grads[1:])
    for rows in (3, 100):  # no hidden elements: a product over nothing
        x = torch.randn(rows, 16, device=DEV)
        out = torch.full_like(x, math.nan)
        q = rsx.feed_forward(x, w[:0], w[:0], d[:, :0], out, keep=True)
        assert (out == 0).all()
        dx = rsx.feed_forward_grad(x, x, w[:0], w[:0], d[:, :0], q.gate, q.up)[0]
        assert (dx == 0).all()
    assert rsx.feed_forward(torch.empty(5, 0, device=DEV), w[:, :0], w[:, :0], d[:0]).out.shape == (5, 0)
    only = rsx.feed_forward_grad(p.out, p.out, w, w, d, p.gate, p.up, inputs=False)
    assert only[0] is None and only[1] is not None
    only = rsx.feed_forward_grad(p.out, p.out, w, w, d, p.gate, p.up, weights=False)
    assert only[1] is None and only[0] is not None


@pytest.mark.parametrize("rows", [4, 200])
@pytest.mark.parametrize("t", [BF16, F32])
def test_feed_forward_nan_stays_in_its_row(rows, t):
    g = gen(9)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, rows, 72, 88, t))
    clean = rsx.feed_forward(x, wg, wu, wd).out.clone()
    x[2, 5] = math.nan
    x[3, 0] = math.inf
    out = rsx.feed_forward(x, wg, wu, wd).out
    assert torch.isnan(out[2]).all()
    assert not torch.isfinite(out[3]).any()
    keep = [i for i in range(rows) if i not in (2, 3)]
    assert same_bits(out[keep], clean[keep])


# ------------------------------- log probabilities from the hidden state
HEAD = [  # rows, vocab, dim, type, tokens, scale, pad, entropy
    (1, 1, 1, F32, torch.int64, 1.0, 0, True), (1, 131, 8, BF16, torch.int32, 1.0, 0, True), (8, 5000, 64, BF16, torch.int64, 1.0, 0, True),
    (3, 33, 7, F16, torch.int64, 2.5, 1, True), (16, 1000, 100, F32, torch.int32, 0.3, 3, False),
    (17, 257, 130, BF16, torch.int64, 1.0, 8, True), (64, 300, 64, F16, torch.int64, 1.0, 0, True),
    (65, 129, 64, BF16, torch.int64, 1.0, 0, True), (66, 1, 40, BF16, torch.int64, 1.0, 0, True),
    (100, 2051, 72, F16, torch.int64, -1.5, 0, True), (129, 1000, 33, F32, torch.int32, 1.0, 1, True),
    (200, 4099, 96, BF16, torch.int64, 1.0, 0, False), (257, 513, 200, F32, torch.int64, 0.5, 0, True),
    (300, 9001, 24, BF16, torch.int64, 4.0, 3, True),
]


def some_tokens(g, rows, vocab, kt):
    t = torch.randint(0, vocab, (rows,), generator=g)
    if rows > 2:
        t[1], t[rows // 2] = -1, vocab
    return t.to(kt)


@pytest.mark.parametrize("rows,vocab,dim,t,kt,scale,pad,ent", HEAD)
def test_linear_logprobs(rows, vocab, dim, t, kt, scale, pad, ent):
    say("linear_logprobs", rows, vocab, dim, t, kt, scale, pad)
    g = gen(rows + vocab)
    h, w = rand(g, rows, dim, dtype=t), rand(g, vocab, dim, dtype=t, scale=2 * dim ** -0.5)
    tok = some_tokens(g, rows, vocab, kt)
    hd, wd, td = place(h, pad)[1], place(w, pad)[1], tok.to(DEV)
    plan = rsx.LinearLogprobs(hd, wd, td, scale)
    plan()
    ref, tol = po.linear_logprobs(h, w, tok, scale)
    for what in ("lse", "logprob", "entropy"):
        so.close(getattr(plan, what), ref[what], tol[what], what)
    once = {k: getattr(plan, k).clone() for k in ("lse", "logprob", "entropy", "lse_rest")}
    plan()
    assert all(same_bits(v, getattr(plan, k)) for k, v in once.items())
    gl, ge = rand(g, rows), rand(g, rows, scale=0.1) if ent else None
    wtype = F32 if rows % 2 else t
    old = rand(g, vocab, dim, dtype=wtype)
    big, dw = wide_rows(old, pad)
    dh_big, dh = wide_rows(torch.zeros(rows, dim, dtype=t), pad)
    lse = plan.lse.cpu().double() + plan.lse_rest.cpu().double()
    hent = plan.entropy.cpu() if ent else None
    (rh, rw), (eh, ew) = po.linear_logprobs_grad(h, w, tok, lse, hent, gl, ge, scale)
    for acc in (False, True):
        rsx.linear_logprobs_grad(hd, wd, td, plan.lse, gl.to(DEV), plan.entropy if ent else None, ge.to(DEV) if ent else None, dh, dw,
                                 lse_rest=plan.lse_rest, scale=scale, accumulate=acc)
        fits(dh, rh, eh, t, "dhidden")
        r, e = (rw, ew) if not acc else (rw + first.double(), ew + 4 * so.U * (rw.abs() + first.double().abs()))  # noqa: F821
        fits(dw, r, e, wtype, "dweight")
        first = dw.cpu()
    assert pad == 0 or (untouched(big, pad, dim) and untouched(dh_big, pad, dim))


@pytest.mark.parametrize("rows,vocab,dim,t", [(2050, 16500, 264, BF16), (40, 100003, 1001, BF16), (3000, 9000, 72, F16), (4097, 40000, 64, BF16),
                                              (20000, 9000, 64, BF16), (333, 70001, 16, F32)])
def test_linear_logprobs_large(rows, vocab, dim, t):
    """Large tiles, and (the fourth and fifth) a vocabulary in pieces, against the logits' own operators in fp64."""
    say("linear_logprobs large", rows, vocab, dim, t)
    g = torch.Generator(device=DEV).manual_seed(rows)
    h = torch.randn(rows, dim, generator=g, device=DEV).to(t)
    w = (torch.randn(vocab, dim, generator=g, device=DEV) * 2 * dim ** -0.5).to(t)
    tok = torch.randint(-1, vocab + 1, (rows,), generator=g, device=DEV)
    p = rsx.linear_logprobs(h, w, tok)
    gl = torch.randn(rows, generator=g, device=DEV)
    dh, dw = rsx.linear_logprobs_grad(h, w, tok, p.lse, gl, lse_rest=p.lse_rest)
    pick = torch.randint(0, rows, (64,), generator=torch.Generator().manual_seed(1))
    ref, tol = po.linear_logprobs(h.cpu()[pick], w.cpu(), tok.cpu()[pick], 1.0)
    for what in ("lse", "logprob", "entropy"):
        so.close(getattr(p, what)[pick.to(DEV)], ref[what], tol[what], what)
    # dz from these lse in 64 bits, a stretch of rows at a time
    rh, rw = torch.empty(rows, dim, dtype=torch.float64, device=DEV), torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
    eh, ew = torch.empty_like(rh), torch.zeros_like(rw)
    lse = p.lse.double() + p.lse_rest.double()
    step = max(1, (1 << 25) // vocab)
    for i in range(0, rows, step):
        s = slice(i, i + step)
        (a, b), (ea, eb) = po.linear_logprobs_grad(h[s], w, tok[s], lse[s], None, gl[s], None, 1.0)
        rh[s], eh[s] = a, ea
        rw += b
        ew += eb
    parts = {BF16: 1, F16: 2, F32: 3}[t]
    ew += po.terms(t, rows, parts) * (rw.abs() + ew)  # sums longer than the stretches'
    assert (dh.double() - rh).abs().le(eh + 1.01 * so.rounding(rh, t)).all()
    assert (dw.double() - rw).abs().le(ew + 1.01 * so.rounding(rw, t)).all()


@pytest.mark.parametrize("rows,vocab", [(6, 300), (80, 300), (2060, 8300)])
def test_linear_logprobs_whole_numbers(rows, vocab):
    """Logits of whole numbers are exact: the same as the operators of given logits make of them, but for the sums' order."""
    g = gen(7)
    dim = 520
    h, w = whole(g, rows, dim, 5).to(DEV, BF16), whole(g, vocab, dim, 200, (-2, -1, 1, 3)).to(DEV, BF16)
    z = h.double() @ w.double().t()
    tok = torch.randint(0, vocab, (rows,), generator=g).to(DEV)
    p = rsx.linear_logprobs(h, w, tok)
    q = rsx.token_logprobs(z.float(), tok)
    n = 2 * (vocab / 256 + 200) * so.U  # the two sums' roundings
    for what in ("lse", "logprob"):
        a, b = getattr(p, what).double(), getattr(q, what).double()
        assert ((a - b).abs() <= n + 8 * so.U * b.abs().clamp(min=20)).all(), what
    assert ((p.entropy - q.entropy).abs() <= 2 * n * 40).all()


@pytest.mark.parametrize("rows", [5, 90])
@pytest.mark.parametrize("t", [BF16, F32])
def test_linear_logprobs_rows_without_a_distribution(rows, t):
    vocab, dim = 200, 16
    h, w = torch.zeros(rows, dim), torch.zeros(vocab, dim)
    w[:, 0] = torch.linspace(-2, 2, vocab)
    w[:, 1] = -1.0
    w[:, 2] = (torch.arange(vocab) != 7).float()
    h[:, 0] = 1.0
    h[1, 3] = math.nan
    h[2, 1] = 1e38
    h[2, 0] = 0
    h, w = h.to(DEV, t), w.to(DEV, t)
    tok = torch.full((rows,), 7, device=DEV)
    p = rsx.linear_logprobs(h, w, tok)
    # NaN in one row alone; logits of -1e38 each are a distribution like any other
    assert all(torch.isnan(getattr(p, k)[1]) for k in ("lse", "logprob", "entropy"))
    good = [i for i in range(rows) if i != 1]
    assert all(torch.isfinite(getattr(p, k)[good]).all() for k in ("lse", "logprob", "entropy"))
    assert abs(p.entropy[2].item() - math.log(vocab)) < 1e-4 and abs(p.logprob[2].item() + math.log(vocab)) < 1e-4
    # one weight of minus infinity masks its token; all of them leave nothing
    w2 = torch.zeros(vocab, 8, device=DEV, dtype=t)
    w2[7, 0] = -math.inf
    h2 = torch.zeros(rows, 8, device=DEV, dtype=t)
    h2[:, 0] = 1
    if t != F32:  # three parts of an infinity times parts of 0 are NaN
        p = rsx.linear_logprobs(h2, w2, tok)
        assert torch.equal(p.logprob, torch.full_like(p.logprob, -math.inf))
        assert (p.lse - math.log(vocab - 1)).abs().max() < 1e-5
        w2[:, 0] = -math.inf
        p = rsx.linear_logprobs(h2, w2, tok)
        assert torch.equal(p.lse, torch.full_like(p.lse, -math.inf)) and torch.equal(p.logprob, p.lse)
        assert (p.entropy == 0).all() and (p.lse_rest == 0).all()
        _, dw = rsx.linear_logprobs_grad(h2, w2, tok, p.lse, torch.ones(rows, device=DEV), inputs=False)
        assert (dw == 0).all()


def test_linear_logprobs_of_nothing():
    w = torch.randn(50, 16, device=DEV)
    none = torch.empty(0, 16, device=DEV)
    tok = torch.empty(0, dtype=torch.int64, device=DEV)
    p = rsx.linear_logprobs(none, w, tok)
    assert p.lse.shape == (0,)
    dh, dw = rsx.linear_logprobs_grad(none, w, tok, p.lse, p.lse)
    assert dh.shape == (0, 16) and (dw == 0).all()
    for rows in (3, 70):  # no dimensions: logits of 0
        p = rsx.linear_logprobs(torch.empty(rows, 0, device=DEV), w[:, :0], torch.zeros(rows, dtype=torch.int32, device=DEV))
        assert (p.lse - math.log(50)).abs().max() < 1e-5 and (p.logprob + math.log(50)).abs().max() < 1e-5


# ------------------------------------------------- orthogonalised updates
ORTHO = [  # shape, type, steps, coefficients, pad
    ((1, 1), F32, 5, po.USUAL, 0), ((1, 7), BF16, 5, po.USUAL, 0), ((9, 1), F16, 3, po.USUAL, 1), ((3, 5, 8), F32, 5, po.USUAL, 0),
    ((64, 64), BF16, 5, po.USUAL, 0), ((65, 130), F32, 5, po.USUAL, 3), ((130, 65), F32, 5, po.USUAL, 1), ((2, 200, 72), F16, 5, po.USUAL, 0),
    ((128, 512), BF16, 5, po.USUAL, 8), ((300, 129), BF16, 1, (1.5, -0.5, 0.0), 0), ((257, 263), F32, 10, (1.875, -1.25, 0.375), 0),
    ((5, 33, 31), F32, 2, (0.0, 1.0, 0.0), 0), ((600, 1000), F32, 5, po.USUAL, 0), ((700, 530), F16, 5, po.USUAL, 0),
]


def stacked(host, pad):
    if pad == 0:
        return host.to(DEV)
    big = torch.full((*host.shape[:-1], host.shape[-1] + 2 * pad), math.nan, dtype=host.dtype, device=DEV)
    view = big[..., pad:pad + host.shape[-1]]
    view.copy_(host)
    return view


def ortho_bound(x, steps, coefficients, t):
    """(result, bound of any element): four times the furthest of three runs with random errors in every rounding."""
    ref = po.newton_schulz(x, steps, coefficients, 1e-7)
    far = max((po.newton_schulz(x, steps, coefficients, 1e-7, torch.Generator().manual_seed(s), t) - ref).abs().max().item() for s in range(3))
    return ref, 4 * far + 2.0 ** -36


@pytest.mark.parametrize("shape,t,steps,coefficients,pad", ORTHO)
def test_newton_schulz(shape, t, steps, coefficients, pad):
    say("newton_schulz", shape, t, steps, coefficients, pad)
    g = gen(sum(shape))
    x = rand(g, *shape, dtype=t, scale=1e-3)
    if min(shape[-2:]) > 8:  # one strong direction
        x = (x + 0.05 * torch.ones(shape[-2], 1) * rand(g, shape[-1])).to(t)
    d = stacked(x, pad)
    plan = rsx.NewtonSchulz(d, steps=steps, coefficients=coefficients)
    plan()
    assert plan.out.is_contiguous() and same_bits(d.cpu().contiguous(), x)
    for one, got in zip(x.reshape(-1, *shape[-2:]), plan.out.reshape(-1, *shape[-2:])):
        ref, tol = ortho_bound(one, steps, coefficients, t)
        fits(got, ref, torch.tensor(tol), t, "out")
    once = plan.out.clone()
    rsx.newton_schulz(d, d, steps=steps, coefficients=coefficients)  # in place
    assert same_bits(d.contiguous(), once)


@pytest.mark.parametrize("rows,cols,batch", [(2100, 4200, 1), (4300, 2050, 1), (1100, 1100, 3), (260, 2000, 2)])
def test_newton_schulz_large(rows, cols, batch):
    say("newton_schulz large", rows, cols, batch)
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(batch, rows, cols, generator=g, device=DEV) * 0.01 + torch.randn(batch, rows, 1, generator=g, device=DEV) * 0.1
    out = rsx.newton_schulz(x)
    for one, got in zip(x, out):
        far = 0.0
        ref = po.newton_schulz(one, 5, po.USUAL, 1e-7)
        noisy = po.newton_schulz(one, 5, po.USUAL, 1e-7, torch.Generator().manual_seed(0))
        far = (noisy - ref).abs().max().item()
        assert ((got.double() - ref).abs() <= 4 * far + 1.01 * so.rounding(ref, F32)).all()


def test_newton_schulz_scale_and_permutation():
    """A permutation has singular values of one size: five steps of the polynomial say what they become."""
    n = 200
    perm = torch.randperm(n, generator=gen(1))
    s = n ** -0.5
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in po.USUAL)
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    for size in (1e-20, 1.0, 1e30):  # squares outside fp32
        x = torch.zeros(n, n)
        x[torch.arange(n), perm] = size
        out = rsx.newton_schulz(x.to(DEV), eps=0.0).cpu().double()
        # each step's relative errors, a few of 2^-22, times how fast the value changes with the one before (a = 3.4445 at most)
        assert (out - s * (x.double() / size)).abs().max() < 5 * 8 * 2.0 ** -22 * 3.4445 ** 5 * s * 0.1


def test_newton_schulz_zeros_and_nan():
    x = torch.zeros(3, 40, 70, device=DEV)
    x[1] = torch.randn(40, 70, generator=gen(2)).to(DEV)
    x[2] = x[1]
    x[2, 3, 4] = math.nan
    out = rsx.newton_schulz(x)
    assert (out[0] == 0).all() and torch.isfinite(out[1]).all() and torch.isnan(out[2]).all()
    assert same_bits(out[1], rsx.newton_schulz(x[1]))
    assert rsx.newton_schulz(x[:0]).shape == (0, 40, 70)
    assert rsx.newton_schulz(x[:, :0]).shape == (3, 0, 70)


# --------------------------------------------- together, streams and graphs
def step_plans(rows, dim, hidden, vocab, t=BF16):
    """A block, its output matrix with the loss, backward through both, and the block's update."""
    g = gen(rows)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, rows, dim, hidden, t))
    w = rand(g, vocab, dim, dtype=t, scale=dim ** -0.5).to(DEV)
    tok = torch.randint(0, vocab, (rows,), generator=g).to(DEV)
    minus = torch.full((rows,), -1.0 / rows, device=DEV)
    ff = rsx.FeedForward(x, wg, wu, wd, keep=True)
    lp = rsx.LinearLogprobs(ff.out, w, tok)
    dlp = rsx.LinearLogprobsGrad(ff.out, w, tok, lp.lse, minus, lse_rest=lp.lse_rest)
    dff = rsx.FeedForwardGrad(dlp.dhidden, x, wg, wu, wd, ff.gate, ff.up)
    ns = rsx.NewtonSchulz(dff.dw_gate)
    plans = [ff, lp, dlp, dff, ns]
    outs = [ff.out, lp.logprob, dlp.dhidden, dlp.dweight, dff.dx, dff.dw_gate, dff.dw_up, dff.dw_down, ns.out]
    return plans, outs, (x, wg, wu, wd, w, tok)


def test_a_step_of_all_of_them():
    plans, outs, (x, wg, wu, wd, w, tok) = step_plans(300, 136, 264, 1000)
    for p in plans:
        p()
    x, wg, wu, wd, w = (m.double().requires_grad_(True) for m in (x, wg, wu, wd, w))
    fn = torch.nn.functional
    y = fn.linear(fn.silu(fn.linear(x, wg)) * fn.linear(x, wu), wd)
    logp = torch.log_softmax(fn.linear(y, w), 1).gather(1, tok[:, None])[:, 0]
    grads = torch.autograd.grad(-logp.mean(), (w, x, wg, wu, wd))
    got = [outs[3], outs[4], outs[5], outs[6], outs[7]]
    for a, b, what in zip(got, grads, ("w", "x", "wg", "wu", "wd")):
        # bf16 operands in a row of five products: 5 roundings of 2^-8 each, of sums that cancel
        assert (a.double() - b).norm() < 5 * 2.0 ** -8 * b.norm(), what
    q = outs[8].double()
    s = torch.linalg.svdvals(q)
    assert 0.6 < s.min() and s.max() < 1.3  # five steps take singular values from 2^-9 of the norm up into this range


@pytest.mark.parametrize("rows", [12, 300])
def test_graph_replays(rows):
    plans, outs, (x, *_rest) = step_plans(rows, 136, 264, 1000)
    for p in plans:
        p()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for p in plans:
            p()
    for turn in range(3):
        x.copy_(torch.randn(x.shape, generator=gen(turn)))
        for p in plans:
            p()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert same_bits(o, v), turn


def test_two_streams_at_once():
    one, two = step_plans(300, 136, 264, 1000), step_plans(260, 200, 96, 777)
    want = []
    for plans, outs, _ in (one, two):
        for p in plans:
            p()
        want.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (plans, outs, _) in (one, two):
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (plans, _o, _i) in zip(streams, (one, two)):
            for p in plans:
                p(s)
    torch.cuda.synchronize()
    for w, (_, outs, _i) in zip(want, (one, two)):
        assert all(same_bits(a, b) for a, b in zip(w, outs))


def test_functions_on_a_stream():
    g = gen(3)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, 90, 40, 56, BF16))
    w, tok = rand(g, 70, 40, dtype=BF16).to(DEV), torch.randint(0, 70, (90,), generator=g).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = rsx.feed_forward(x, wg, wu, wd, stream=s).out
    b = rsx.linear_logprobs(x, w, tok, stream=s)
    c = rsx.newton_schulz(wg, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert same_bits(a, rsx.feed_forward(x, wg, wu, wd).out)
    assert same_bits(b.logprob, rsx.linear_logprobs(x, w, tok).logprob)
    assert same_bits(c, rsx.newton_schulz(wg))


def test_expanded_inputs_and_refusals():
    g = gen(6)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, 80, 40, 56, BF16))
    row = x[:1].expand(80, 40)
    a = rsx.feed_forward(row, wg, wu, wd).out
    assert same_bits(a, rsx.feed_forward(row.contiguous(), wg, wu, wd).out)
    tok = torch.zeros(80, dtype=torch.int64, device=DEV)
    assert same_bits(rsx.linear_logprobs(row, wg, tok).lse, rsx.linear_logprobs(row.contiguous(), wg, tok).lse)
    with pytest.raises(ValueError, match="shape"):
        rsx.FeedForward(x, wg, wu[:, :32], wd)
    with pytest.raises(ValueError, match="activation"):
        rsx.FeedForward(x, wg, wu, wd, activation="tanh")
    with pytest.raises(ValueError, match="dtype"):
        rsx.FeedForward(x, wg.float(), wu, wd)
    with pytest.raises(ValueError, match="side by side"):
        rsx.FeedForward(x, wg, wu, wd.t().contiguous().t())
    with pytest.raises(rsx.RsxError, match="ALIASING"):
        rsx.feed_forward(x, wg, wu, wd, out=x)
    p = rsx.feed_forward(x, wg, wu, wd, keep=True)
    with pytest.raises(ValueError, match="accumulate"):
        rsx.FeedForwardGrad(x, x, wg, wu, wd, p.gate, p.up, accumulate=True)
    with pytest.raises(ValueError, match="gate"):
        rsx.FeedForwardGrad(x, x, wg, wu, wd, p.gate[:, :8], p.up)
    with pytest.raises(ValueError, match="dw_up has dtype"):
        rsx.FeedForwardGrad(x, x, wg, wu, wd, p.gate, p.up, dw_up=torch.empty(56, 40, dtype=F16, device=DEV))
    with pytest.raises(ValueError, match="dtype"):
        rsx.LinearLogprobs(x, wg.to(F16), tok)
    with pytest.raises(ValueError, match="no rows"):
        rsx.LinearLogprobs(x, wg[:0], tok)
    with pytest.raises(ValueError, match="finite"):
        rsx.LinearLogprobs(x, wg, tok, scale=math.inf)
    with pytest.raises(ValueError, match="tokens has shape"):
        rsx.LinearLogprobs(x, wg, tok[:4])
    with pytest.raises(ValueError, match="entropy"):
        rsx.LinearLogprobsGrad(x, wg, tok, a[:, 0].float(), a[:, 0].float(), dentropy=a[:, 0].float())
    with pytest.raises(ValueError, match="steps"):
        rsx.NewtonSchulz(wg, steps=0)
    with pytest.raises(ValueError, match="two dimensions"):
        rsx.NewtonSchulz(wg[0])
    with pytest.raises(ValueError, match="side by side"):
        rsx.NewtonSchulz(wg.t())
    with pytest.raises(ValueError, match="overlap"):
        rsx.NewtonSchulz(wg, wg[:1].expand(56, 40))


def block_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_example_gradients():
    vocab, dim, hidden, tokens = 203, 72, 136, 301
    r = block_example().Rank(vocab, dim, hidden, tokens, seed=3, dtype=F32)
    r.next_batch()
    loss = r.gradients()
    table, weight, bias, proj, wg, wu, wd = params = [p.double().requires_grad_(True) for p in r.params]
    fn = torch.nn.functional
    x = fn.embedding(r.tokens, table) * dim ** 0.5
    y = fn.layer_norm(x, (dim,), weight, bias, 1e-5)
    z = fn.linear(x + fn.linear(fn.silu(fn.linear(y, wg)) * fn.linear(y, wu), wd), proj) * dim ** -0.5
    want = -torch.log_softmax(z, 1).gather(1, r.targets[:, None]).mean()
    # ten operators in a row, sums of at most `tokens` values with a rounding of fp32 each
    tol = 10 * tokens * 2.0 ** -24
    assert abs(loss.item() - want.item()) < tol * want.item()
    for what, a, b in zip(r.NAMES, r.grads, torch.autograd.grad(want, params)):
        assert (a.double() - b).norm() < tol * b.norm(), what


def test_example_runs_and_its_ranks_agree():
    losses, world = block_example().train(ranks=3, steps=4, vocab=200, dim=64, hidden=96, tokens=500)
    assert all(math.isfinite(v) for v in losses)
    for r in world[1:]:
        assert all(same_bits(p, q) for p, q in zip(r.params, world[0].params))
        assert all(torch.isfinite(p).all() for p in r.params)


def test_both_projections_gradients_have_strides_of_their_own():
    """dw_gate and dw_up come from one launch: unlike strides and addresses, alone and added to."""
    g = gen(9)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, 90, 40, 56, BF16))
    dout = rand(g, 90, 40).to(BF16).to(DEV)
    p = rsx.feed_forward(x, wg, wu, wd, keep=True)
    want = rsx.feed_forward_grad(dout, x, wg, wu, wd, p.gate, p.up)
    for accumulate in (False, True):
        bufs = [torch.full((56, 40 + pad), math.nan, dtype=BF16, device=DEV) for pad in (3, 11)]
        views = [bufs[0][:, 1:41], bufs[1][:, 8:48]]
        for v in views:
            v.zero_()
        down = torch.zeros(40, 56, dtype=BF16, device=DEV)
        rsx.feed_forward_grad(dout, x, wg, wu, wd, p.gate, p.up, dw_gate=views[0], dw_up=views[1], dw_down=down, accumulate=accumulate)
        # 0 + v is v, of either sign (an exact 0 may differ in its sign)
        assert all(torch.equal(a, b) for a, b in zip((*views, down), want[1:]))
        assert all(torch.isnan(b).sum() == 56 * (b.shape[1] - 40) for b in bufs)


@pytest.mark.parametrize("rows,dim,hidden,t,act,pad,keep", [
    # 2^14 values and more of few rows, in one part: k uncut, cut, with ends off the vectors, and just on either side
    (8, 2056, 200, BF16, "silu", 0, True), (16, 1024, 4100, F16, "gelu", 0, False), (31, 1001, 2050, BF16, "relu", 1, False),
    (32, 513, 2100, F16, "silu", 8, True), (16, 1023, 130, BF16, "gelu_tanh", 0, False), (33, 496, 72, BF16, "silu", 0, False),
    (33, 497, 72, F16, "silu", 3, False), (64, 300, 2100, BF16, "gelu", 1, True)])
def test_feed_forward_few_rows_of_many(rows, dim, hidden, t, act, pad, keep):
    test_feed_forward(rows, dim, hidden, t, act, pad, keep)


@pytest.mark.parametrize("rows,dim,hidden", [(5, 270, 192), (29, 24, 7101), (2, 40, 5000), (40, 300, 200), (100, 24, 1000)])
def test_small_results_are_as_good_as_their_rounding(rows, dim, hidden):
    say("small results", rows, dim, hidden)
    host = block(gen(rows + dim), rows, dim, hidden, BF16)
    out = rsx.feed_forward(*(h.to(DEV) for h in host)).out
    # the bounds of matrices kept whole, and what two bf16 parts of s leave out: a half step of the second, 2^-9 of 2^-9
    ref, tol = po.feed_forward(*(h.float() for h in host), "silu")
    x, wg, wu, wd = (h.double() for h in host)
    g = x @ wg.t()
    s = g * torch.sigmoid(g) * (x @ wu.t())
    fits(out, ref[0], tol[0] + 2.0 ** -17 * (s.abs() @ wd.abs().t()), BF16, "out")
