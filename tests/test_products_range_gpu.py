"""The step's matrix products on the GPU at the ends of their ranges: what is no number, and what is not asked for."""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
from parity_util import say
from test_products_gpu import block
from test_steps_gpu import BF16, DEV, F16, F32, gen, rand, same_bits

pytestmark = pytest.mark.gpu


def gradients(host, dy, act, spoil=None):
    """(out, dx, dw_gate, dw_up, dw_down) of the block, one of its matrices spoilt."""
    x, wg, wu, wd = (m.to(DEV) for m in host)
    if spoil is not None:
        spoil(x, wg, wu, wd)
    p = rsx.feed_forward(x, wg, wu, wd, activation=act, keep=True)
    return (p.out, *rsx.feed_forward_grad(dy.to(DEV), x, wg, wu, wd, p.gate, p.up, activation=act))


@pytest.mark.parametrize("act", sorted(rsx.ACTIVATIONS))
@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("rows,dim,hidden", [(4, 72, 88), (70, 136, 40), (300, 264, 520)])
def test_nan_shows_in_every_gradient(rows, dim, hidden, t, act):
    say("nan in gradients", rows, dim, hidden, t, act)
    g = gen(rows + dim)
    host, dy = block(g, rows, dim, hidden, t), rand(g, rows, dim, dtype=t)
    clean = gradients(host, dy, act)
    r = hidden // 2

    def gate_row(x, wg, wu, wd):
        wg[r, dim // 3] = math.nan
    out, dx, dg, du, dd = gradients(host, dy, act, gate_row)
    # the row's gate is NaN for all rows of x
    for what, got, spoilt, want in (("dw_gate", dg, dg[r], clean[2]), ("dw_up", du, du[r], clean[3]), ("dw_down", dd.t(), dd[:, r], clean[4].t())):
        assert torch.isnan(spoilt).all(), what
        rest = [i for i in range(hidden) if i != r]
        assert same_bits(got[rest].contiguous(), want[rest].contiguous()), what
    assert torch.isnan(out).all() and torch.isnan(dx).all()

    def input_row(x, wg, wu, wd):
        x[1, dim // 2] = math.nan
    out, dx, dg, du, dd = gradients(host, dy, act, input_row)
    rest = [i for i in range(rows) if i != 1]
    assert torch.isnan(out[1]).all() and torch.isnan(dx[1]).all()
    assert same_bits(out[rest], clean[0][rest]) and same_bits(dx[rest], clean[1][rest])
    assert all(torch.isnan(d).all() for d in (dg, du, dd))


@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("rows,vocab,dim", [(5, 300, 40), (90, 131, 72), (600, 4100, 136)])
def test_rows_without_a_gradient_add_nothing(rows, vocab, dim, t):
    """Padding of a batch: rows whose token is none of the vocabulary, or whose gradients are 0, whatever they hold."""
    say("rows without a gradient", rows, vocab, dim, t)
    g = gen(rows)
    h, w = rand(g, rows, dim, dtype=t).to(DEV), rand(g, vocab, dim, dtype=t, scale=dim ** -0.5).to(DEV)
    tok = torch.randint(0, vocab, (rows,), generator=g).to(DEV)
    gl, ge = rand(g, rows).to(DEV), rand(g, rows, scale=0.1).to(DEV)
    tok[1], tok[3] = -1, vocab
    gl[4] = 0.0  # a loss mask
    ge[[1, 3, 4]] = 0.0
    h[[1, 3, 4]] = 0.0
    for entropy in (False, True):
        def grads():
            p = rsx.linear_logprobs(h, w, tok)
            return p, *rsx.linear_logprobs_grad(h, w, tok, p.lse, gl, p.entropy if entropy else None, ge if entropy else None,
                                                lse_rest=p.lse_rest)
        h[[1, 3, 4]] = 0.0
        _, dh, dw = grads()
        h[1], h[3, 2], h[4] = math.nan, math.inf, -math.inf
        p, dh2, dw2 = grads()
        assert torch.isnan(p.lse[1]) and torch.isfinite(dw).all()
        assert (dh2[[1, 3, 4]] == 0).all()
        assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
        h[0, 0] = math.nan  # a row with a gradient shows
        _, dh3, dw3 = grads()
        assert torch.isnan(dh3[0]).all() and torch.isnan(dw3).all()
        h[0, 0] = 0.5
