"""The step's matrix products on the GPU at the ends of their ranges: what is no number, and what is not asked for."""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
import product_digits as pd
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


def same_kind(got, ref, what):
    """NaN, either infinity and numbers in the same places."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    for inf in (math.inf, -math.inf):
        assert torch.equal(got == inf, ref == inf), what


@pytest.mark.parametrize("rows,dim,hidden", [(4, 72, 88), (70, 136, 40), (300, 264, 520)])
@pytest.mark.parametrize("where", ["x", "w_gate", "w_down", "dout"])
def test_fp32_infinities_are_those_of_the_products(rows, dim, hidden, where):
    """In parts too: no part of a finite value times an infinity may be a NaN or an infinity of the other sign."""
    say("fp32 infinities", rows, dim, hidden, where)
    g = gen(rows + 1)
    host, dy = block(g, rows, dim, hidden, F32), rand(g, rows, dim)
    x, wg, wu, wd = host
    at = {"x": x, "w_gate": wg, "w_down": wd, "dout": dy}[where]
    at[1, 5], at[2, 7] = math.inf, -math.inf
    x[3, 5] = 0.0  # times an infinity: NaN
    dev = [m.to(DEV) for m in host]
    p = rsx.feed_forward(*dev, activation="relu", keep=True)
    x, wg, wu, wd, dy64 = (m.double() for m in (*host, dy))
    gate, up = x @ wg.t(), x @ wu.t()
    same_kind(p.gate.cpu(), gate, "gate")
    same_kind(p.up.cpu(), up, "up")
    act = torch.where(gate < 0, 0.0, gate)
    same_kind(p.out.cpu(), (act * up) @ wd.t(), "out")
    ds = dy64 @ wd
    dg, du = ds * up * torch.where(gate.isnan(), gate, (gate > 0).double()), ds * act
    grads = rsx.feed_forward_grad(dy.to(DEV), *dev, p.gate, p.up, activation="relu")
    for got, ref, what in zip(grads, (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, dy64.t() @ (act * up)), ("dx", "dw_gate", "dw_up", "dw_down")):
        same_kind(got.cpu(), ref, what)


@pytest.mark.parametrize("rows", [3, 80])
def test_fp32_values_past_the_largest_bf16_one(rows):
    dim, hidden = 24, 40
    x, w = torch.zeros(rows, dim, device=DEV), torch.zeros(hidden, dim, device=DEV)
    x[:, 3] = torch.finfo(F32).max
    x[1, 3] = -torch.finfo(F32).max
    w[:, 3] = 2.0 ** -torch.arange(hidden, device=DEV)
    p = rsx.feed_forward(x, w, w * 2.0 ** -60, torch.zeros(dim, hidden, device=DEV), activation="relu", keep=True)
    assert torch.equal(p.gate, x[:, 3:4] * w[:, 3])


@pytest.mark.parametrize("rows,vocab,dim", [(5, 200, 40), (66, 131, 24), (90, 1000, 72), (600, 4100, 136)])
def test_fp32_masks(rows, vocab, dim):
    """A weight of minus infinity masks its token, with few rows and with many."""
    say("fp32 masks", rows, vocab, dim)
    g = gen(rows + vocab)
    h, w = rand(g, rows, dim), rand(g, vocab, dim, scale=dim ** -0.5)
    h[:, 3] = h[:, 3].abs() + 0.1
    masked = torch.randperm(vocab, generator=g)[:vocab // 3]
    w[masked, 3] = -math.inf
    tok = torch.randint(0, vocab, (rows,), generator=g)
    tok[0] = masked[0]
    logp = torch.log_softmax(h.double() @ w.double().t(), 1)
    p = rsx.linear_logprobs(h.to(DEV), w.to(DEV), tok.to(DEV))
    want = logp.gather(1, tok[:, None])[:, 0]
    got = p.logprob.cpu().double()
    assert torch.equal(got == -math.inf, want == -math.inf)
    some = torch.isfinite(want)
    # logits of size 1 from sums of `dim` products, six parts' each, with a whole step for every addition
    assert (got - want)[some].abs().max() < 2.0 ** -23 * (6 * dim + 64) * 4
    assert torch.isfinite(p.lse).all() and torch.isfinite(p.entropy).all()
    gl = rand(g, rows)
    gl[tok == masked[0]] = 0.0
    _, dw = rsx.linear_logprobs_grad(h.to(DEV), w.to(DEV), tok.to(DEV), p.lse, gl.to(DEV), lse_rest=p.lse_rest, inputs=False)
    assert torch.isfinite(dw).all()
    clear = masked[~torch.isin(masked, tok)]
    assert (dw[clear.to(DEV)] == 0).all()
    w[:, 3] = -math.inf
    p = rsx.linear_logprobs(h.to(DEV), w.to(DEV), tok.to(DEV))
    assert (p.lse == -math.inf).all() and (p.logprob == -math.inf).all() and (p.entropy == 0).all()


@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("rows,cols,batch", [(72, 40, 3), (40, 136, 2), (300, 257, 2)])
def test_updates_side_by_side(rows, cols, batch, t):
    """The slices of a fused projection: matrices that lie in the same rows."""
    say("updates side by side", rows, cols, batch, t)
    g = gen(rows)
    x = rand(g, batch, rows, cols, dtype=t, scale=1e-3).to(DEV)
    want = rsx.newton_schulz(x)
    wide = torch.full((rows, batch * cols + 5), math.nan, dtype=t, device=DEV)
    wide[:, 3:3 + batch * cols] = x.transpose(0, 1).reshape(rows, batch * cols)
    side = wide[:, 3:3 + batch * cols].unflatten(1, (batch, cols)).transpose(0, 1)
    assert same_bits(rsx.newton_schulz(side), want)
    other = torch.full_like(wide, math.nan)
    to = other[:, 1:1 + batch * cols].unflatten(1, (batch, cols)).transpose(0, 1)
    rsx.newton_schulz(side, to)
    assert same_bits(to.contiguous(), want) and torch.isnan(other).sum() == 5 * rows
    rsx.newton_schulz(side, side)
    assert same_bits(side.contiguous(), want) and torch.isnan(wide).sum() == 5 * rows
    with pytest.raises(ValueError, match="overlap"):
        rsx.NewtonSchulz(wide.as_strided((batch, rows, cols), (cols - 1, batch * cols + 5, 1)))


@pytest.mark.parametrize("rows,dim,hidden,names", pd.BLOCKS)
def test_fp32_block_keeps_its_digits(rows, dim, hidden, names):
    say("fp32 digits", rows, dim, hidden, names)
    inputs = pd.block_inputs(rows, dim, hidden, names)
    ref, bound = pd.block(*inputs, names), pd.block_bounds(rows, dim, hidden)
    x, wg, wu, wd, dy, gate, up = (m.to(DEV) for m in inputs)
    p = rsx.feed_forward(x, wg, wu, wd, activation="relu", keep=True)
    dx, dg, du, dd = rsx.feed_forward_grad(dy, x, wg, wu, wd, gate, up, activation="relu")
    got = {"gate": p.gate, "up": p.up, "out": p.out, "dx": dx, "dw_gate": dg, "dw_up": du, "dw_down": dd}
    for n in names:
        far = pd.off(got[n], ref[n])
        print(n, f"{far / pd.U:.2f} of {bound[n] / pd.U:.2f} half steps")
        assert far <= bound[n], n


@pytest.mark.parametrize("rows,vocab,dim,name", pd.HEADS)
def test_fp32_head_keeps_its_digits(rows, vocab, dim, name):
    say("fp32 digits", rows, vocab, dim, name)
    inputs = pd.head_inputs(rows, vocab, dim, name)
    ref, bound = pd.head(*inputs, name), pd.head_bounds(rows, vocab, dim)[name]
    h, w, tok, gl, ge = (None if m is None else m.to(DEV) for m in inputs)
    p = rsx.linear_logprobs(h, w, tok)
    got = {"logprob": p.logprob}
    if ge is not None:
        got["dhidden"], got["dweight"] = rsx.linear_logprobs_grad(h, w, tok, p.lse, gl, p.entropy, ge, lse_rest=p.lse_rest)
    far = pd.head_off(name, got[name], ref)
    print(f"{far / pd.U:.2f} of {bound / pd.U:.2f} half steps")
    assert far <= bound


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("dim,hidden", [(4096, 264), (1024, 4100), (264, 520), (40, 5000), (512, 511), (512, 512)])
def test_a_row_has_the_same_digits_in_any_call(dim, hidden, t):
    """How an operand is rounded does not depend on how many rows share the call."""
    say("same digits", dim, hidden, t)
    g = gen(dim)
    x, wg, wu, wd = (m.to(DEV) for m in block(g, 300, dim, hidden, t))
    few = rsx.feed_forward(x[:16], wg, wu, wd).out
    for rows in (1, 2, 3, 4, 7, 15):
        assert same_bits(rsx.feed_forward(x[:rows], wg, wu, wd).out, few[:rows]), rows
    # sums of another order, 64 bits' results of the two rules for s
    g64, u64, wd64 = x.double() @ wg.double().t(), x.double() @ wu.double().t(), wd.double()
    s = g64 * torch.sigmoid(g64) * u64
    whole, once = s @ wd64.t(), s.to(t).double() @ wd64.t()
    rounding = (whole.to(t).double() - whole).square().mean().sqrt()
    for rows in (16, 40, 300):
        off = (rsx.feed_forward(x[:rows], wg, wu, wd).out.double() - whole[:rows]).square().mean().sqrt()
        apart = (once - whole)[:rows].square().mean().sqrt()
        # two parts leave the result's rounding, one adds its own; a tenth for what is random in either
        want = rounding if dim * hidden < 1 << 18 else torch.hypot(rounding, apart)
        assert 0.9 * want < off < 1.1 * want, rows
