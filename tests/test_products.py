"""The step's matrix products without a GPU: refusals, sizes, and the oracle.

Calls with made-up addresses have to be refused before any HIP call; they are
skipped where a GPU is visible.
"""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
from collective_reduction_ring_amd import _lib as L
import product_oracle as po
import step_oracle as so
from test_abi import fake_ptrs
from test_steps import A, ALIAS, BAD, BF16, BIG, F16, F32, I32, I64, I8, OK, TYPE, UNSUPPORTED, _differences, call

OP = 3
MB = 1 << 20


def ffn(x=A(1), xs=64, g=A(2), gs=64, u=A(3), us=64, d=A(4), ds=96, out=A(5), os=64, kg=A(6), ku=A(7), rows=80, dim=64, hidden=96,
        act=0, t=BF16, ws=A(8), wb=16 * MB):
    return call("rsx_feed_forward", x, xs, g, gs, u, us, d, ds, out, os, kg, ku, rows, dim, hidden, act, t, ws, wb)


def ffn_grad(dy=A(1), ys=64, x=A(2), xs=64, g=A(3), gs=64, u=A(4), us=64, d=A(5), ds=96, kg=A(6), ku=A(7), dx=A(8), dxs=64, dg=A(9),
             dgs=64, du=A(10), dus=64, dd=A(11), dds=96, rows=80, dim=64, hidden=96, act=0, t=BF16, wt=BF16, acc=0, ws=A(12),
             wb=16 * MB):
    return call("rsx_feed_forward_grad", dy, ys, x, xs, g, gs, u, us, d, ds, kg, ku, dx, dxs, dg, dgs, du, dus, dd, dds, rows, dim,
                hidden, act, t, wt, acc, ws, wb)


def head(h=A(1), hs=64, w=A(2), wst=64, t=BF16, tok=A(3), kt=I64, rows=80, vocab=300, dim=64, lp=A(4), ent=A(5), lse=A(6), rest=A(7),
         ws=A(8), wb=16 * MB):
    return call("rsx_linear_logprobs", h, hs, w, wst, t, tok, kt, rows, vocab, dim, 1.0, lp, ent, lse, rest, ws, wb)


def head_grad(h=A(1), hs=64, w=A(2), wst=64, t=BF16, tok=A(3), kt=I64, lse=A(4), rest=A(5), ent=A(6), g=A(7), d=A(8), dh=A(9), dhs=64,
              dw=A(10), dws=64, wt=BF16, acc=0, rows=80, vocab=300, dim=64, ws=A(11), wb=16 * MB):
    return call("rsx_linear_logprobs_grad", h, hs, w, wst, t, tok, kt, lse, rest, ent, g, d, dh, dhs, dw, dws, wt, acc, rows, vocab, dim,
                1.0, ws, wb)


def ortho(x=A(1), xs=64, xm=6400, out=A(2), os=64, om=6400, batch=2, rows=100, cols=64, steps=5, eps=1e-7, t=BF16, ws=A(3), wb=16 * MB):
    return call("rsx_newton_schulz", x, xs, xm, out, os, om, batch, rows, cols, steps, 3.4, -4.8, 2.0, eps, t, ws, wb)


W = 1 << 22
REFUSALS = [
    (ffn, dict(t=I32), TYPE), (ffn, dict(act=4), OP), (ffn, dict(act=-1), OP), (ffn, dict(x=None), BAD), (ffn, dict(g=None), BAD),
    (ffn, dict(u=None), BAD), (ffn, dict(d=None), BAD), (ffn, dict(out=None), BAD), (ffn, dict(kg=None), BAD), (ffn, dict(ku=None), BAD),
    (ffn, dict(xs=63), BAD), (ffn, dict(ds=95), BAD), (ffn, dict(os=0), BAD), (ffn, dict(x=A(1) + 1), BAD), (ffn, dict(ws=None), BAD),
    (ffn, dict(wb=100), BAD), (ffn, dict(ws=A(8) + 128), BAD), (ffn, dict(out=A(1)), ALIAS), (ffn, dict(out=A(2) + 64), ALIAS),
    (ffn, dict(kg=A(7)), ALIAS), (ffn, dict(kg=A(5)), ALIAS), (ffn, dict(ws=A(4)), ALIAS), (ffn, dict(rows=BIG), UNSUPPORTED),
    (ffn, dict(dim=W, xs=W, gs=W, us=W, os=W), UNSUPPORTED), (ffn, dict(hidden=W, ds=W), UNSUPPORTED),
    (ffn, dict(xs=1 << 45), UNSUPPORTED),
    (ffn_grad, dict(t=I8), TYPE), (ffn_grad, dict(wt=F16), TYPE), (ffn_grad, dict(wt=I32), TYPE), (ffn_grad, dict(act=7), OP),
    (ffn_grad, dict(dy=None), BAD), (ffn_grad, dict(kg=None), BAD), (ffn_grad, dict(ku=None), BAD), (ffn_grad, dict(dg=None), BAD),
    (ffn_grad, dict(dd=None), BAD), (ffn_grad, dict(dxs=63), BAD), (ffn_grad, dict(dds=95), BAD), (ffn_grad, dict(wb=4096), BAD),
    (ffn_grad, dict(ws=None), BAD), (ffn_grad, dict(dx=A(1)), ALIAS), (ffn_grad, dict(dx=A(2)), ALIAS), (ffn_grad, dict(dg=A(3)), ALIAS),
    (ffn_grad, dict(dg=A(10)), ALIAS), (ffn_grad, dict(dd=A(8) + 64), ALIAS), (ffn_grad, dict(ws=A(6)), ALIAS),
    (ffn_grad, dict(rows=BIG), UNSUPPORTED), (ffn_grad, dict(dim=W, ys=W, xs=W, gs=W, us=W, dxs=W, dgs=W, dus=W), UNSUPPORTED),
    (head, dict(t=I32), TYPE), (head, dict(kt=F32), TYPE), (head, dict(h=None), BAD), (head, dict(w=None), BAD), (head, dict(tok=None), BAD),
    (head, dict(lp=None), BAD), (head, dict(lse=None), BAD), (head, dict(vocab=0), BAD), (head, dict(hs=32), BAD), (head, dict(wst=32), BAD),
    (head, dict(ws=None), BAD), (head, dict(wb=1000), BAD), (head, dict(lp=A(5)), ALIAS), (head, dict(lse=A(1)), ALIAS),
    (head, dict(rest=A(3)), ALIAS), (head, dict(ws=A(2)), ALIAS), (head, dict(vocab=BIG), UNSUPPORTED), (head, dict(rows=BIG), UNSUPPORTED),
    (head, dict(dim=W, hs=W, wst=W), UNSUPPORTED), (head, dict(rows=BIG - 1, vocab=BIG - 1), UNSUPPORTED),
    (head_grad, dict(t=I64), TYPE), (head_grad, dict(wt=F16), TYPE), (head_grad, dict(kt=BF16), TYPE), (head_grad, dict(lse=None), BAD),
    (head_grad, dict(g=None), BAD), (head_grad, dict(ent=None), BAD), (head_grad, dict(vocab=0), BAD), (head_grad, dict(dhs=63), BAD),
    (head_grad, dict(dws=63), BAD), (head_grad, dict(ws=None), BAD), (head_grad, dict(wb=4096), BAD), (head_grad, dict(dh=A(1)), ALIAS),
    (head_grad, dict(dw=A(2)), ALIAS), (head_grad, dict(dw=A(9)), ALIAS), (head_grad, dict(ws=A(8)), ALIAS),
    (head_grad, dict(rows=BIG), UNSUPPORTED), (head_grad, dict(vocab=BIG), UNSUPPORTED),
    (ortho, dict(t=I32), TYPE), (ortho, dict(steps=0), BAD), (ortho, dict(eps=-1.0), BAD), (ortho, dict(eps=math.nan), BAD),
    (ortho, dict(x=None), BAD), (ortho, dict(out=None), BAD), (ortho, dict(xs=32), BAD), (ortho, dict(os=32), BAD), (ortho, dict(os=0), BAD),
    (ortho, dict(om=6399), BAD), (ortho, dict(ws=None), BAD), (ortho, dict(wb=4096), BAD), (ortho, dict(out=A(1) + 2), ALIAS),
    (ortho, dict(out=A(1), om=6500), ALIAS), (ortho, dict(out=A(1), os=65, om=6500), ALIAS), (ortho, dict(ws=A(1)), ALIAS),
    (ortho, dict(batch=1 << 16), UNSUPPORTED), (ortho, dict(cols=W, xs=W, os=W), UNSUPPORTED), (ortho, dict(rows=W), UNSUPPORTED),
    (ortho, dict(xm=1 << 60), UNSUPPORTED),
]


@fake_ptrs
@pytest.mark.parametrize("fn,kw,want", REFUSALS, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_refusals(fn, kw, want):
    assert fn(**kw) == want


@fake_ptrs
@pytest.mark.parametrize("fn,kw", [(ffn, dict(rows=0)), (ffn, dict(dim=0)), (ffn_grad, dict(dim=0)),
                                   (ffn_grad, dict(dx=None, dg=None, du=None, dd=None)), (head, dict(rows=0)), (head_grad, dict(dim=0)),
                                   (head_grad, dict(dh=None, dw=None)), (ortho, dict(batch=0)), (ortho, dict(rows=0)),
                                   (ortho, dict(cols=0))],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_nothing_to_do(fn, kw):
    assert fn(**kw) == OK


@fake_ptrs
def test_matrices_that_are_copied_need_room():
    lib = L.lib()
    small = lib.rsx_feed_forward_workspace_size(80, 64, 96, BF16, 0)
    large = lib.rsx_feed_forward_workspace_size(80, 64, 96, BF16, 1)
    assert small < large
    assert ffn(wb=small - 1) == BAD
    for odd in (dict(x=A(1) + 2), dict(gs=65), dict(d=A(4) + 8, ds=97), dict(us=0)):
        assert ffn(wb=large - 1, **odd) == BAD, odd
    small, large = (lib.rsx_linear_logprobs_grad_workspace_size(80, 300, 64, BF16, c) for c in (0, 1))
    assert small < large
    assert head_grad(wb=large - 1, w=A(2) + 2) == BAD


def test_workspace_sizes():
    lib = L.lib()
    n, d, f = 8192, 4096, 11008
    # the product between the two layers
    need = lib.rsx_feed_forward_workspace_size(n, d, f, BF16, 0)
    assert n * f * 2 <= need <= n * f * 2 + 256 * 256 * 256 * 4 + (1 << 16)
    # three of them, no copies, and the sums of cut tiles: at most 256 KB of fp32 for each of 256 CUs
    cut = 256 * 256 * 256 * 4
    need = lib.rsx_feed_forward_grad_workspace_size(n, d, f, BF16, 0)
    assert 3 * n * f * 2 <= need <= 3 * n * f * 2 + cut + (1 << 16)
    # nothing of the size of the logits
    v = 131072
    assert lib.rsx_linear_logprobs_workspace_size(n, v, d, BF16, 0) < n * v // 4
    assert lib.rsx_linear_logprobs_grad_workspace_size(n, v, d, BF16, 0) < n * v * 2 // 3
    assert lib.rsx_linear_logprobs_workspace_size(0, v, d, BF16, 0) == 0
    assert lib.rsx_linear_logprobs_workspace_size(8, v, W, BF16, 0) == 0
    assert lib.rsx_feed_forward_workspace_size(8, d, f, I32, 0) == 0
    # two matrices and two squares of 4 bytes an element
    need = lib.rsx_newton_schulz_workspace_size(2, 4096, 1024)
    assert 2 * 2 * 4 * (4096 * 1024 + 1024 * 1024) <= need <= 2 * 2 * 4 * (4096 * 1024 + 1024 * 1024) + cut + (1 << 16)
    assert lib.rsx_newton_schulz_workspace_size(0, 64, 64) == 0


def test_python_refuses():
    x, w, d, t = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(8, 6), torch.zeros(4, dtype=torch.int64)
    for make in (lambda: rsx.FeedForward(x, w, w, d), lambda: rsx.FeedForwardGrad(x, x, w, w, d, x, x),
                 lambda: rsx.LinearLogprobs(x, w, t), lambda: rsx.LinearLogprobsGrad(x, w, t, x, x), lambda: rsx.NewtonSchulz(x),
                 lambda: rsx.newton_schulz(x, stream=0)):
        with pytest.raises(ValueError, match="not on a GPU"):
            make()
    with pytest.raises(TypeError):
        rsx.NewtonSchulz([1.0])


def test_header_constants():
    import os
    import re
    text = open(os.path.join(os.path.dirname(L.PKG), "include", "rsx.h")).read()
    for name, value in rsx.ACTIVATIONS.items():
        assert int(re.search(rf"RSX_ACT_{name.upper()} = (\d+)", text).group(1)) == value


# ---- the oracle against differences and against torch in 64 bits
@pytest.mark.parametrize("act", sorted(rsx.ACTIVATIONS))
def test_oracle_feed_forward(act):
    g = torch.Generator().manual_seed(3)
    x, wg, wu, wd, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 5), (7, 5), (7, 5), (5, 7), (3, 5)))
    fn = torch.nn.functional
    want = {"silu": fn.silu, "relu": fn.relu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh")}[act]
    (y, gate, up), _ = po.feed_forward(x, wg, wu, wd, act)
    assert (y - fn.linear(want(fn.linear(x, wg)) * fn.linear(x, wu), wd)).abs().max() < 1e-12
    grads, _ = po.feed_forward_grad(dy, x, wg, wu, wd, gate, up, act)
    # differences of step 1e-5 in 64 bits: about 1e-10 of the step's square, 1e-10 of rounding
    args = [x, wg, wu, wd]
    for i, got in enumerate(grads):
        f = lambda v, i=i: (po.feed_forward(*args[:i], v, *args[i + 1:], act)[0][0] * dy).sum()  # noqa: E731
        assert (got - _differences(f, args[i])).abs().max() < 1e-6, i


def test_oracle_linear_logprobs():
    g = torch.Generator().manual_seed(4)
    h, w = torch.randn(4, 6, generator=g, dtype=torch.float64), torch.randn(9, 6, generator=g, dtype=torch.float64)
    tok = torch.tensor([3, -1, 8, 0])
    gl, gh = torch.randn(4, generator=g, dtype=torch.float64), torch.randn(4, generator=g, dtype=torch.float64)
    scale = 0.75  # a power of two's multiple: the same in 32 bits

    def f(h, w):
        o = so.token_logprobs(scale * (h @ w.t()), tok, 0)[0]
        return (o["logprob"] * gl + o["entropy"] * gh).sum()
    z, _ = po.logits(h.float(), w.float(), scale)
    assert (z - scale * (h.float().double() @ w.float().double().t())).abs().max() < 1e-12
    o = so.token_logprobs(scale * (h @ w.t()), tok, 0)[0]
    hf, wf = h.float().double(), w.float().double()
    o = so.token_logprobs(scale * (hf @ wf.t()), tok, 0)[0]
    (dh, dw), _ = po.linear_logprobs_grad(h.float(), w.float(), tok, o["lse"], o["entropy"], gl, gh, scale)
    assert (dh - _differences(lambda v: f(v, wf), hf)).abs().max() < 1e-6
    assert (dw - _differences(lambda v: f(hf, v), wf)).abs().max() < 1e-6


def test_oracle_newton_schulz():
    """Against the singular values, each taken through the polynomial by itself."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, 9, generator=g, dtype=torch.float64)
    u, s, vh = torch.linalg.svd(x / x.norm(), full_matrices=False)
    a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in po.USUAL)
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    want = (u * s) @ vh
    got = po.newton_schulz(x, 5, po.USUAL, 0.0)
    assert (got - want).abs().max() < 1e-10
    assert (po.newton_schulz(x.t(), 5, po.USUAL, 0.0) - want.t()).abs().max() < 1e-10
    assert (s > 0.6).all() and (s < 1.3).all()


@pytest.mark.parametrize("t", [BF16, F16, F32])
def test_a_workspace_for_copies_is_right_without(t):
    lib = L.lib()
    for rows in (1, 16, 17, 32, 33, 64, 65, 300):
        for dim, hidden in ((64, 96), (4096, 11008), (128, 40000), (7, 5)):
            for size, args in ((lib.rsx_feed_forward_workspace_size, (rows, dim, hidden)),
                               (lib.rsx_feed_forward_grad_workspace_size, (rows, dim, hidden)),
                               (lib.rsx_linear_logprobs_workspace_size, (rows, hidden, dim)),
                               (lib.rsx_linear_logprobs_grad_workspace_size, (rows, hidden, dim))):
                assert size(*args, t, 0) <= size(*args, t, 1), (size.__name__, args)
