"""The training-step operators on the GPU against their definitions in 64 bits.

Bounds come from step_oracle: they count the fp32 roundings of a sum, plus the
one rounding to the output's type.
"""
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
import step_oracle as so
from parity_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def wide_rows(host, pad, fill=math.nan, dtype=None):
    """`host` on the GPU as a column slice of a wider matrix, `pad` columns on either side."""
    r, d = host.shape
    dtype = host.dtype if dtype is None else dtype
    big = torch.full((r, d + 2 * pad), fill, dtype=dtype, device=DEV)
    view = big[:, pad:pad + d]
    view.copy_(host)
    return big, view


def untouched(big, pad, d, fill=None):
    edge = torch.cat([big[:, :pad], big[:, pad + d:]], 1)
    return bool(torch.isnan(edge).all()) if fill is None else bool((edge == fill).all())


def same_bits(a, b):
    w = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(w), b.contiguous().view(w))


# --------------------------------------------------------------- embedding
EMBED = [  # n, vocab, dim, table, out, tokens, first, pad
    (1, 1, 1, F32, F32, torch.int64, 0, 0), (3, 17, 5, BF16, F32, torch.int32, 0, 1), (65, 300, 64, F16, BF16, torch.int64, 0, 0),
    (7, 100, 511, BF16, BF16, torch.int64, 40, 3), (33, 1000, 2049, F32, BF16, torch.int32, 0, 0),
    (4, 50, 8192, F32, F32, torch.int64, -20, 0), (2100, 64, 2056, BF16, F16, torch.int64, 0, 4),
    (1111, 70, 4001, F16, F16, torch.int32, 0, 0), (1, 9, 16385, F32, F16, torch.int64, 0, 0),
]


@pytest.mark.parametrize("n,vocab,dim,tt,ot,kt,first,pad", EMBED)
def test_embedding(n, vocab, dim, tt, ot, kt, first, pad):
    g = gen(n + dim)
    table = rand(g, vocab, dim, dtype=tt)
    tok = torch.randint(first - 2, first + vocab + 2, (n,), generator=g).to(kt)
    say("embedding", n, vocab, dim, tt, ot, kt, first, pad)
    _, t = wide_rows(table, pad)
    big, out = wide_rows(torch.zeros(n, dim, dtype=ot), pad)
    rsx.embedding(t, tok.to(DEV), out, scale=1.7, first=first)
    # one product in fp32 and one rounding: the same bits as torch's
    idx = tok.long() - first
    ok = (idx >= 0) & (idx < vocab)
    want = torch.where(ok[:, None], table[idx.clamp(0, vocab - 1)].float() * torch.tensor(1.7), 0.0).to(ot)
    assert torch.equal(out.cpu(), want)
    assert pad == 0 or untouched(big, pad, dim)
    ref = so.embedding(table, tok, 1.7, first)
    so.close(out, ref, so.U * ref.abs() + 1.01 * so.rounding(ref, ot), "embedding")


def test_embedding_far_tokens_and_shapes():
    table = torch.arange(12.0, device=DEV).view(4, 3)
    tok = torch.tensor([[2 ** 62, -2 ** 62, 3], [-1, 4, 0]], device=DEV)
    out = rsx.embedding(table, tok)
    assert out.shape == (2, 3, 3)
    assert out[0, 2].tolist() == [9, 10, 11] and out[1, 2].tolist() == [0, 1, 2]
    assert out[0, :2].abs().sum() == 0 and out[1, :2].abs().sum() == 0
    # a difference that leaves 64 bits behind is outside too
    assert rsx.embedding(table, torch.tensor([-2 ** 63, 2 ** 63 - 1], device=DEV), first=5).abs().sum() == 0
    assert rsx.embedding(table, torch.empty(0, 2, dtype=torch.int32, device=DEV)).shape == (0, 2, 3)
    assert rsx.embedding(table[:0], tok).abs().sum() == 0


GRAD = [  # n, vocab, dim, dout, grad, tokens, first, kind, accumulate, pad
    (0, 5, 7, F32, F32, torch.int64, 0, "any", False, 0), (1, 1, 1, F32, F32, torch.int64, 0, "any", False, 0),
    (1, 3, 9, BF16, F32, torch.int32, 0, "any", True, 2), (64, 64, 64, BF16, BF16, torch.int64, 0, "any", False, 0),
    (100, 1000, 33, F16, F32, torch.int32, 100, "any", False, 1), (8191, 513, 65, BF16, F32, torch.int64, 0, "zipf", False, 0),
    (8192, 512, 40, F32, F32, torch.int64, 0, "one", False, 0), (8193, 511, 24, BF16, BF16, torch.int32, 0, "zipf", True, 0),
    (20000, 100003, 17, F16, F16, torch.int64, 7, "zipf", False, 3), (50001, 300000, 8, BF16, F32, torch.int64, 0, "any", False, 0),
    (40000, 70, 520, BF16, F32, torch.int64, 0, "one", False, 0), (3000, 200, 1030, F32, BF16, torch.int32, 0, "sorted", False, 0),
    (600, 40, 4097, BF16, BF16, torch.int64, 0, "outside", False, 0), (9000, 64, 16, F32, F16, torch.int64, 0, "few", True, 0),
    (32, 40, 300, BF16, F32, torch.int64, 0, "few", False, 0), (33, 9000, 72, F32, F32, torch.int64, 0, "any", False, 1),
    (140001, 3001, 24, BF16, F32, torch.int64, 5, "zipf", False, 1), (131073, 520, 9, F32, BF16, torch.int32, 0, "few", False, 0),
    (131072, 5000, 10, F16, F32, torch.int64, -3, "zipf", False, 0), (10, 70000, 2, F32, BF16, torch.int64, 0, "any", False, 0),
    (9001, 600000, 1, BF16, BF16, torch.int64, 0, "zipf", False, 0), (70000, 2000, 1100, BF16, BF16, torch.int64, 0, "zipf", False, 0),
    (128, 77, 30, F16, F16, torch.int64, 0, "few", False, 0), (129, 77, 30, F16, F16, torch.int64, 0, "few", False, 1),
    (70001, 3, 30, F32, BF16, torch.int64, 0, "any", False, 0), (30001, 900, 4, BF16, F32, torch.int32, 0, "one", True, 0),
    (65537, 2 ** 20, 11, BF16, BF16, torch.int64, 0, "zipf", False, 0), (8193, 40000, 3, F16, F16, torch.int64, -7, "any", False, 0),
    (5568, 32831, 66, BF16, BF16, torch.int64, 0, "zipf", False, 0), (124, 25216, 507, BF16, BF16, torch.int64, 0, "any", False, 0),
    (3, 72576, 263, F16, F32, torch.int64, 0, "any", False, 0), (20, 5001, 7, F16, F16, torch.int32, 0, "any", False, 0),
    (700, 900, 3, F32, F32, torch.int64, 0, "any", False, 0), (129, 100001, 1, BF16, BF16, torch.int64, 0, "any", False, 0),
    (512, 700, 300, BF16, BF16, torch.int64, 0, "zipf", False, 0), (513, 700, 300, BF16, BF16, torch.int64, 0, "zipf", False, 0),
    (512, 1, 1030, F16, F32, torch.int64, 0, "one", False, 0), (257, 9, 8200, BF16, BF16, torch.int32, 0, "few", False, 1),
    (511, 3000, 5, F32, F16, torch.int64, 9, "few", True, 3), (512, 40, 4100, F32, F32, torch.int64, 0, "one", True, 0),
    (64, 300, 2, BF16, F32, torch.int64, 0, "one", False, 1), (65, 20, 515, BF16, F32, torch.int64, 0, "sorted", False, 0),
    (400, 65, 77, BF16, BF16, torch.int64, 0, "outside", False, 0), (0, 3000, 33, F32, BF16, torch.int64, 0, "any", False, 1),
    (321, 40000, 16, BF16, F32, torch.int32, -4, "zipf", False, 0), (7, 600000, 16, F32, F32, torch.int64, 0, "any", False, 0),
    (2, 3, 40000, F32, F32, torch.int64, 0, "any", False, 0), (512, 90, 2048, BF16, BF16, torch.int64, 0, "zipf", False, 0),
    (512, 90, 2049, BF16, BF16, torch.int64, 0, "zipf", False, 0), (160, 70, 9001, BF16, F32, torch.int64, 0, "any", False, 0),
    (520, 65, 40, BF16, BF16, torch.int64, 0, "outside", False, 0),
]


def draw_tokens(g, n, vocab, first, kind):
    if kind == "zipf":
        t = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
        return (t * 48271 + 3) % vocab + first
    if kind == "one":
        return torch.full((n,), vocab // 2 + first)
    if kind == "sorted":
        return torch.arange(n) * vocab // max(n, 1) + first
    if kind == "outside":
        return torch.full((n,), first - 1)
    if kind == "few":
        return torch.randint(0, 3, (n,), generator=g) * (vocab // 3) + first
    return torch.randint(first - 1, first + vocab + 1, (n,), generator=g)


@pytest.mark.parametrize("n,vocab,dim,dt,gt,kt,first,kind,acc,pad", GRAD)
def test_embedding_grad(n, vocab, dim, dt, gt, kt, first, kind, acc, pad):
    g = gen(n + dim)
    dout = rand(g, n, dim, dtype=dt)
    tok = draw_tokens(g, n, vocab, first, kind).to(kt)
    old = rand(g, vocab, dim, dtype=gt)
    say("embedding_grad", n, vocab, dim, dt, gt, kt, first, kind, acc, pad)
    _, d = wide_rows(dout, pad)
    big, grad = wide_rows(old, pad)
    plan = rsx.EmbeddingGrad(d, tok.to(DEV), grad, scale=0.37, first=first, accumulate=acc)
    plan()
    ref, tol = so.embedding_grad(dout, tok, vocab, 0.37, first, old if acc else None)
    so.close(grad, ref, tol + 1.01 * so.rounding(ref, gt), "grad")
    assert pad == 0 or untouched(big, pad, dim)
    once = grad.clone()
    grad.copy_(old)
    plan()
    assert same_bits(once, grad)  # one order of the sums


@pytest.mark.parametrize("shift", [1, 3, 7])
@pytest.mark.parametrize("n,vocab,dim,gt", [(50, 3001, 33, BF16), (50, 3001, 33, F32), (900, 700, 5, F16), (9000, 20001, 9, BF16)])
def test_embedding_grad_of_a_table_off_its_boundary(n, vocab, dim, gt, shift):
    g = gen(n + shift)
    flat = torch.full((vocab * dim + 16,), math.nan, dtype=gt, device=DEV)
    grad = flat[shift:shift + vocab * dim].view(vocab, dim)
    d, tok = rand(g, n, dim), torch.randint(0, vocab, (n,), generator=g)
    say("embedding_grad off a boundary", n, vocab, dim, gt, shift)
    rsx.embedding_grad(d.to(DEV), tok.to(DEV), grad)
    ref, tol = so.embedding_grad(d, tok, vocab, 1.0, 0)
    so.close(grad, ref, tol + 1.01 * so.rounding(ref, gt), "grad")
    assert torch.isnan(flat[:shift]).all() and torch.isnan(flat[shift + vocab * dim:]).all()


def test_embedding_grad_rows_beyond_32_bits():
    # a table of more than 2^32 elements; only the rows named are looked at
    vocab, dim = 1_100_003, 4000
    grad = torch.empty(vocab, dim, dtype=BF16, device=DEV)
    tok = torch.tensor([vocab - 1, 5, vocab - 1, 1_080_000], device=DEV)
    d = torch.ones(4, dim, dtype=BF16, device=DEV)
    say("embedding_grad beyond 2^32 elements")
    rsx.embedding_grad(d, tok, grad)
    assert (grad[-1] == 2).all() and (grad[5] == 1).all() and (grad[1_080_000] == 1).all()
    assert (grad[-2] == 0).all() and (grad[1_079_999] == 0).all() and (grad[1_099_000] == 0).all()
    out = rsx.embedding(grad, tok, scale=0.5)
    assert (out[0] == 1).all() and (out[1] == 0.5).all()


def test_sharded_embedding_sums_to_the_whole_table():
    """A table cut over W = 4 ranks: lookup by part, sum all-reduce; the gradient by part."""
    g = gen(5)
    table, tok = rand(g, 403, 96), torch.randint(0, 403, (50,), generator=g)
    cuts = [0, 101, 202, 303, 403]
    t, k = table.to(DEV), tok.to(DEV)
    outs = [rsx.embedding(t[a:b].contiguous(), k, first=a) for a, b in zip(cuts, cuts[1:])]
    rsx.all_reduce(outs, None, "sum")
    whole = rsx.embedding(t, k)
    for o in outs:
        assert torch.equal(o, whole)
    d = rand(g, 50, 96).to(DEV)
    full = rsx.embedding_grad(d, k, torch.empty_like(t))
    parts = [rsx.embedding_grad(d, k, torch.empty(b - a, 96, device=DEV), first=a) for a, b in zip(cuts, cuts[1:])]
    assert same_bits(torch.cat(parts), full)


# -------------------------------------------------------------- layer norm
NORM = [  # rows, dim, x, weight, pad, affine
    (1, 1, F32, F32, 0, "wb"), (3, 2, BF16, BF16, 1, "wb"), (5, 31, F32, F32, 1, "wb"), (7, 33, F16, F32, 0, "w"),
    (2, 512, BF16, F32, 0, "wb"), (9, 513, BF16, BF16, 3, ""), (4, 2047, F32, F32, 0, "wb"), (3, 2049, F16, F16, 1, "b"),
    (2, 4096, BF16, BF16, 0, "wb"), (3, 8191, BF16, F32, 0, "wb"), (2, 16383, F32, F32, 2, "wb"), (2, 16385, BF16, BF16, 0, "wb"),
    (2, 32768, F32, F32, 0, "wb"), (2, 33001, F16, F32, 1, "wb"), (2, 70001, F32, F32, 0, "w"),
    (2048, 100, BF16, BF16, 0, "wb"), (2051, 600, F32, F32, 0, "wb"), (2050, 1111, F16, F16, 1, "wb"),
    (2049, 2056, BF16, F32, 0, "wb"), (2048, 4096, F32, F32, 0, "wb"),
    (4097, 40, BF16, F32, 0, "wb"), (4099, 255, F32, F32, 1, "wb"), (4101, 511, F16, F16, 0, "w"), (4097, 1030, BF16, BF16, 0, "b"),
    (4097, 2050, F16, F32, 1, "wb"), (3, 9001, BF16, F32, 0, "wb"), (2, 12287, F32, F32, 1, "wb"), (2, 8, BF16, BF16, 0, "wb"),
]


def norm_inputs(g, rows, dim, xt, wt, affine):
    x = rand(g, rows, dim, dtype=xt, scale=2.0, shift=1.5)
    w = rand(g, dim, dtype=wt, scale=0.3, shift=1.0) if "w" in affine else None
    b = rand(g, dim, dtype=wt, scale=0.3) if "b" in affine else None
    return x, w, b


@pytest.mark.parametrize("rows,dim,xt,wt,pad,affine", NORM)
def test_layer_norm(rows, dim, xt, wt, pad, affine):
    g = gen(rows + dim)
    x, w, b = norm_inputs(g, rows, dim, xt, wt, affine)
    say("layer_norm", rows, dim, xt, wt, pad, affine)
    _, xd = wide_rows(x, pad)
    big, y = wide_rows(torch.zeros(rows, dim, dtype=xt), pad)
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    ck = rsx.Checkpoint(x.shape, DEV)
    plan = rsx.LayerNorm(xd, on(w), on(b), y, eps=1e-5, checkpoint=ck)
    plan()
    (ry, rm, rr), (ty, tm, tr) = so.layer_norm(x, w, b, 1e-5)
    so.close(plan.mean, rm, tm + 1.01 * so.rounding(rm, F32), "mean")
    so.close(plan.rstd, rr, tr + 1.01 * so.rounding(rr, F32), "rstd")
    so.close(y, ry, ty + 1.01 * so.rounding(ry, xt), "y")
    assert pad == 0 or untouched(big, pad, dim)
    codes, scales = so.checkpoint(x)
    assert torch.equal(ck.codes.cpu(), codes) and torch.equal(ck.scales.cpu(), scales)
    # in place, and without a checkpoint: the same bits
    want = y.clone()
    rsx.layer_norm(xd, on(w), on(b), xd, eps=1e-5)
    assert same_bits(xd, want)


def test_layer_norm_rows_that_are_special():
    x = torch.zeros(6, 300)
    x[1] = 1e4                      # no variance: rstd = eps^-1/2 of an exact zero
    x[2, 7] = math.nan
    x[3, 11] = math.inf
    x[4] = torch.arange(300) * 1e18  # large, finite squares' sum
    x[5] = torch.arange(300) * 1e-30
    y, mean, rstd = rsx.layer_norm(x.to(DEV))
    y, rstd = y.cpu(), rstd.cpu()
    assert (y[0] == 0).all() and (y[1] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    (ry, _, _), (ty, _, _) = so.layer_norm(x[4:5], None, None, 1e-5)
    so.close(y[4:5], ry, ty + so.rounding(ry, F32))
    assert (y[5].abs() < 1e-24).all() and abs(rstd[0].item() - 1e-5 ** -0.5) < 1e-4


NGRAD = [  # rows, dim, x, weight, pad, affine
    (1, 1, F32, F32, 0, "w"), (3, 2, BF16, BF16, 1, "w"), (5, 31, F32, F32, 1, "w"), (7, 33, F16, F32, 0, ""),
    (130, 512, BF16, F32, 0, "w"), (9, 513, BF16, BF16, 3, "w"), (601, 1000, F16, F16, 0, "w"), (4, 2047, F32, F32, 0, "w"),
    (3, 2049, F16, F16, 1, "w"), (1200, 1025, BF16, BF16, 0, "w"), (515, 4096, BF16, BF16, 0, "w"), (3, 8191, BF16, F32, 0, "w"),
    (520, 8192, F32, F32, 0, "w"), (2, 16383, F32, F32, 2, "w"), (514, 12000, BF16, BF16, 0, "w"), (3, 16385, BF16, BF16, 0, "w"),
    (513, 20001, F32, F32, 1, "w"), (2100, 96, BF16, F32, 0, "w"),
    (16385, 16, BF16, F32, 0, "w"), (8193, 129, F32, F32, 1, "w"), (4097, 300, F16, F16, 0, ""), (1025, 2047, F32, F32, 0, "w"),
    (513, 8191, BF16, BF16, 1, "w"), (514, 16380, F32, F32, 0, "w"), (2, 8, BF16, BF16, 0, "w"),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,dim,xt,wt,pad,affine", NGRAD)
def test_layer_norm_grad(rows, dim, xt, wt, pad, affine, packed):
    g = gen(rows + dim)
    x, w, _ = norm_inputs(g, rows, dim, xt, wt, affine)
    dy = rand(g, rows, dim, dtype=xt)
    (_, mean, rstd), _ = so.layer_norm(x, None, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    say("layer_norm_grad", rows, dim, xt, wt, pad, affine, packed)
    _, xd = wide_rows(x, pad)
    _, dyd = wide_rows(dy, pad)
    big, dx = wide_rows(torch.zeros(rows, dim, dtype=xt), pad)
    wd = None if w is None else w.to(DEV)
    back = x
    src = xd
    if packed:
        src = rsx.checkpoint_pack(xd)
        back = so.checkpoint_values(src.codes, src.scales)
    dw0 = torch.full((dim,), math.nan, dtype=wt if w is not None else xt, device=DEV)
    plan = rsx.LayerNormGrad(dyd, src, mean.to(DEV), rstd.to(DEV), wd, dx, dw0)
    plan()
    ref, tol = so.layer_norm_grad(dy, back, mean, rstd, w)
    for got, r, t, what in zip((dx, plan.dweight, plan.dbias), ref, tol, ("dx", "dweight", "dbias")):
        so.close(got, r, t + 1.01 * so.rounding(r, got.dtype), what)
    assert pad == 0 or untouched(big, pad, dim)
    want = [dx.clone(), plan.dweight.clone(), plan.dbias.clone()]
    plan()
    assert all(same_bits(a, b) for a, b in zip(want, (dx, plan.dweight, plan.dbias)))
    # in the gradient's own place, without the weights
    _, none_w, none_b = rsx.layer_norm_grad(dyd, src, mean.to(DEV), rstd.to(DEV), wd, dyd, weights=False)
    assert none_w is None and none_b is None and same_bits(dyd, want[0])


def test_layer_norm_grad_against_differences():
    g = gen(3)
    x, w, b, dy = (torch.randn(s, generator=g, dtype=torch.float64).float() for s in ((4, 24), (24,), (24,), (4, 24)))
    y, mean, rstd = rsx.layer_norm(x.to(DEV), w.to(DEV), b.to(DEV))
    dx, dw, db = rsx.layer_norm_grad(dy.to(DEV), x.to(DEV), mean, rstd, w.to(DEV))
    f = lambda x, w: (so.layer_norm(x, w, b, 1e-5)[0][0] * dy.double()).sum().item()  # noqa: E731
    h = 1e-5
    for got, at in ((dx, 0), (dw, 1)):
        base = [x.double(), w.double()]
        for i in range(0, base[at].numel(), 5):
            lo, hi = base[at].clone().view(-1), base[at].clone().view(-1)
            lo[i] -= h
            hi[i] += h
            args = lambda v: [v.view_as(base[at]) if k == at else base[k] for k in (0, 1)]  # noqa: E731
            slope = (f(*args(hi)) - f(*args(lo))) / (2 * h)
            # fp32 sums of 24 terms of size about 5: 24 * 2^-24 * 5; differences to 1e-8
            assert abs(got.view(-1)[i].item() - slope) < 24 * so.U * 16 + 1e-7


def test_layer_norm_grad_without_rows_and_with_expanded_rows():
    e = torch.empty(0, 40, device=DEV)
    v = torch.empty(0, device=DEV)
    dx, dw, db = rsx.layer_norm_grad(e, e, v, v, torch.ones(40, device=DEV))
    assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()
    # the gradient of a sum over rows: one row for all
    g = gen(9)
    x, row = rand(g, 37, 50), rand(g, 1, 50)
    y, mean, rstd = rsx.layer_norm(x.to(DEV))
    a = rsx.layer_norm_grad(row.to(DEV).expand(37, 50), x.to(DEV), mean, rstd)
    b = rsx.layer_norm_grad(row.expand(37, 50).contiguous().to(DEV), x.to(DEV), mean, rstd)
    assert all(same_bits(p, q) for p, q in zip(a, b))


# ------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("rows,dim,xt,pad", [(1, 1, F32, 0), (3, 31, BF16, 1), (5, 32, F16, 0), (4, 33, F32, 1), (700, 8, BF16, 0),
                                             (33, 100, F32, 0), (9, 511, BF16, 3), (6, 1025, F16, 0), (2, 70003, BF16, 0),
                                             (300, 4096, BF16, 0), (2049, 1030, F32, 1), (700, 6001, BF16, 0), (301, 8000, F16, 3),
                                             (70001, 33, BF16, 0), (300001, 7, F32, 0), (129, 16400, F32, 0), (2, 8, BF16, 0)])
def test_checkpoint(rows, dim, xt, pad):
    g = gen(rows + dim)
    x = rand(g, rows, dim, dtype=xt) * torch.exp(torch.randn(rows, 1, generator=g) * 3).to(xt)
    x.view(-1)[::7] = 0
    x[-1, :min(dim, 32)] = 0
    say("checkpoint", rows, dim, xt, pad)
    _, xd = wide_rows(x, pad)
    big, out = wide_rows(torch.zeros(rows, dim, dtype=xt), pad)
    c = rsx.checkpoint_pack(xd)
    rsx.checkpoint_unpack(c, out)
    codes, scales = so.checkpoint(x)
    assert torch.equal(c.codes.cpu(), codes) and torch.equal(c.scales.cpu(), scales)
    want = so.checkpoint_values(codes, scales)
    assert torch.equal(out.cpu(), want.to(xt))
    assert torch.equal(rsx.checkpoint_unpack(c).cpu().double(), want)
    assert pad == 0 or untouched(big, pad, dim)
    # an element is off by half a step, or by one where its code is clamped
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)[:, :dim]
    off = (want - x.double()).abs()
    assert (off <= torch.where(codes.abs() == 127, 1.0, 0.5) * step).all()


def test_checkpoint_of_extremes():
    x = torch.zeros(1, 32 * 9)
    b = x.view(9, 32)
    b[0, 3] = math.nan
    b[1, 4], b[1, 5] = math.inf, 1.0
    b[2, 0], b[2, 1] = 3.4028234663852886e38, -1e38   # the type's largest
    b[3, 0], b[3, 1] = 2.0 ** -149, 0.0                # its smallest
    b[4, 0], b[4, 1] = 2.0 ** -121, 2.0 ** -127
    b[5, 0], b[5, 1] = 1.9999999, 1.0                  # clamped
    b[6, 0] = -0.0
    b[7, :] = 1e-38
    b[8, 0], b[8, 1] = 2.0 ** -119, -2.0 ** -126
    c = rsx.checkpoint_pack(x.to(DEV))
    codes, scales = so.checkpoint(x)
    assert torch.equal(c.scales.cpu(), scales)
    assert torch.equal(c.codes.cpu()[:, 64:], codes[:, 64:])
    got = rsx.checkpoint_unpack(c).cpu().view(9, 32)
    assert torch.isnan(got[:2]).all()
    assert torch.equal(got[2:].double(), so.checkpoint_values(codes, scales).view(9, 32)[2:])


# --------------------------------------------------- token log probabilities
LOGP = [  # rows, vocab, top, type, tokens, pad
    (1, 1, 1, F32, torch.int64, 0), (3, 2, 2, BF16, torch.int32, 1), (5, 63, 5, F16, torch.int64, 0), (4, 64, 64, F32, torch.int64, 0),
    (2, 65, 8, BF16, torch.int64, 3), (7, 1000, 0, F32, torch.int32, 0), (3, 2047, 16, BF16, torch.int64, 1),
    (2, 8191, 3, F16, torch.int64, 0), (2, 8193, 64, BF16, torch.int64, 0), (1, 50021, 20, F32, torch.int64, 0),
    (8, 131072, 8, BF16, torch.int64, 0), (1, 262144, 64, BF16, torch.int32, 0), (1030, 777, 4, BF16, torch.int64, 0),
    (300, 20003, 7, BF16, torch.int64, 1), (1, 600000, 1, F16, torch.int64, 0),
    (1025, 7, 3, F32, torch.int64, 1), (1024, 4096, 8, F16, torch.int64, 0), (1024, 4093, 0, BF16, torch.int32, 1),
    (5, 8191, 10, BF16, torch.int64, 5), (2, 16389, 2, F32, torch.int64, 3),
]


def logits(g, rows, vocab, dtype, kind=0):
    z = rand(g, rows, vocab, scale=2.0)
    z[:, torch.rand(vocab, generator=g) < 0.05] = -math.inf
    z[::3, ::2] = -math.inf
    z[:, vocab // 2] = torch.randn(rows, generator=g) * 6  # every row has one
    return z.to(dtype)


@pytest.mark.parametrize("rows,vocab,top,zt,kt,pad", LOGP)
def test_token_logprobs(rows, vocab, top, zt, kt, pad):
    g = gen(rows + vocab)
    z = logits(g, rows, vocab, zt)
    tok = torch.randint(-1, vocab + 1, (rows,), generator=g).to(kt)
    gl, gh = torch.randn(rows, generator=g), torch.randn(rows, generator=g) * 0.1
    say("token_logprobs", rows, vocab, top, zt, kt, pad)
    _, zd = wide_rows(z, pad)
    td = tok.to(DEV)
    p = rsx.token_logprobs(zd, td, top)
    ref, tol = so.token_logprobs(z, tok, top)
    for k, r in ref.items():
        got = getattr(p, k)
        if k == "top_token":
            assert torch.equal(got.cpu(), r), k
        else:
            so.close(got, r, tol[k] + 1.01 * so.rounding(r, F32), k)
    for dent in (gh, None):
        ent = p.entropy.cpu() if dent is not None else None
        big, dz = wide_rows(torch.zeros(rows, vocab, dtype=zt), pad)
        rsx.token_logprobs_grad(zd, td, p.lse, gl.to(DEV), None if dent is None else p.entropy,
                                None if dent is None else dent.to(DEV), dz)
        rz, tz = so.token_logprobs_grad(z, tok, p.lse.cpu(), ent, gl, dent)
        so.close(dz, rz, tz + 1.01 * so.rounding(rz, zt), "dlogits")
        assert pad == 0 or untouched(big, pad, vocab)
    rsx.token_logprobs_grad(zd, td, p.lse, gl.to(DEV), dlogits=zd)
    assert same_bits(zd, dz)


@pytest.mark.parametrize("zt", [F32, BF16])
@pytest.mark.parametrize("vocab,rows", [(9000, 6), (70000, 6), (300, 1200)])
def test_token_logprobs_far_rows(vocab, rows, zt):
    """Logits near the ends of the type's range, some of them only in parts of a row; large ones shift nothing."""
    top = torch.finfo(zt).max
    z = torch.zeros(rows, vocab, dtype=torch.float64)
    z[0] = -top
    z[0, ::2] = -math.inf                             # the lowest beside masked ones
    z[1, vocab // 3:] = -top                          # whole slices of the lowest
    z[2] = torch.where(torch.arange(vocab) % 5 == 0, top, -top)
    z[3] = torch.arange(vocab) % 7 + 2.0 ** 14        # large and close
    z[4, :vocab // 2] = -math.inf                     # whole slices masked
    z[5] = torch.randn(vocab, generator=gen(vocab)) * 1e4
    z = z.to(zt)
    tok = torch.arange(rows) % 3
    say("token_logprobs far", vocab, rows, zt)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV), 3)
    ref, tol = so.token_logprobs(z, tok, 3)
    for k, r in ref.items():
        got = getattr(p, k)
        if k == "top_token":
            assert torch.equal(got.cpu(), r), k
        else:
            so.close(got, r, tol[k] + 1.01 * so.rounding(r, F32), k)


@pytest.mark.parametrize("zt", TYPES)
@pytest.mark.parametrize("vocab", [40, 9000, 70000])
def test_token_logprobs_special_rows(vocab, zt):
    low = torch.finfo(zt).min
    z = torch.zeros(9, vocab)
    z[0] = -math.inf                                  # nothing left
    z[1] = low                                        # masked with the type's lowest: every token alike
    z[2] = low
    z[2, vocab - 3] = 1.0                             # one left among the lowest
    z[3] = -math.inf
    z[3, 5] = 2.0                                     # certain
    z[4, 9] = math.nan
    z[5, vocab // 2] = math.inf
    z[6] = torch.arange(vocab) % 4                    # many ties
    z[7, 1], z[7, 0], z[7, 2] = -0.0, 0.0, -0.0       # zeros of either sign are equal
    z[8] = math.nan
    z = z.to(zt)
    tok = torch.tensor([3, 2, vocab - 3, 5, 0, 1, 2, 7, 1])
    say("token_logprobs special", vocab, zt)
    zd, td = z.to(DEV), tok.to(DEV)
    p = rsx.token_logprobs(zd, td, 6)
    ref, tol = so.token_logprobs(z, tok, 6)
    for k, r in ref.items():
        got = getattr(p, k)
        if k == "top_token":
            assert torch.equal(got.cpu(), r), (k, got.cpu(), r)
        else:
            so.close(got, r, tol[k] + 1.01 * so.rounding(r, F32), k)
    g, h = torch.ones(9), torch.full((9,), 0.5)
    dz = rsx.token_logprobs_grad(zd, td, p.lse, g.to(DEV), p.entropy, h.to(DEV))
    assert (dz[0] == 0).all()
    assert torch.isnan(dz[4]).all() and torch.isnan(dz[5]).all() and torch.isnan(dz[8]).all()
    fine = [0, 1, 2, 3, 6, 7]
    rz, tz = so.token_logprobs_grad(z[fine], tok[fine], p.lse.cpu()[fine], p.entropy.cpu()[fine], g[fine], h[fine])
    so.close(dz[fine], rz, tz + 1.01 * so.rounding(rz, zt), "dlogits")


@pytest.mark.parametrize("zt", [F32, F16])
@pytest.mark.parametrize("rows,vocab,top", [(3, 30001, 64), (4, 2000, 17), (1100, 1500, 33), (2, 200000, 16)])
def test_alternatives_among_equals_and_rising_rows(rows, vocab, top, zt):
    g = gen(vocab)
    z = torch.randint(0, 4, (rows, vocab), generator=g).float()   # thousands of equals
    z[0] = torch.arange(vocab) / 64                                # each step beats the last (in fp16 with equals)
    z[1] = -z[0]
    z[2 % rows, ::3] = -math.inf
    z = z.to(zt)
    tok = torch.zeros(rows, dtype=torch.int64)
    say("alternatives", rows, vocab, top, zt)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV), top)
    ref, tol = so.token_logprobs(z, tok, top)
    assert torch.equal(p.top_token.cpu(), ref["top_token"])
    so.close(p.top_logprob, ref["top_logprob"], tol["top_logprob"] + 1.01 * so.rounding(ref["top_logprob"], F32))
    z[:, 5:9] = math.nan                                           # NaNs come last, and few numbers before them
    z[:, top // 2 + 9:] = math.nan
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV), top)
    assert torch.equal(p.top_token.cpu(), so.token_logprobs(z, tok, top)[0]["top_token"])


def test_token_logprobs_grad_against_differences():
    g = gen(4)
    z = torch.randn(3, 11, generator=g)
    tok = torch.tensor([2, 10, -100])
    gl, gh = torch.randn(3, generator=g), torch.randn(3, generator=g)
    p = rsx.token_logprobs(z.to(DEV), tok.to(DEV))
    dz = rsx.token_logprobs_grad(z.to(DEV), tok.to(DEV), p.lse, gl.to(DEV), p.entropy, gh.to(DEV)).cpu()

    def f(v):
        o = so.token_logprobs(v, tok, 0)[0]
        return (o["logprob"] * gl.double() + o["entropy"] * gh.double()).sum().item()
    h = 1e-5
    for i in range(33):
        lo, hi = z.double().clone().view(-1), z.double().clone().view(-1)
        lo[i] -= h
        hi[i] += h
        slope = (f(hi.view(3, 11)) - f(lo.view(3, 11))) / (2 * h)
        # a dozen fp32 roundings of values up to about 8
        assert abs(dz.view(-1)[i].item() - slope) < 12 * so.U * 8 + 1e-7


def test_logits_rows_beyond_32_bits():
    stride, vocab = (1 << 31) + 8, 1000
    flat = torch.empty(2 * stride + vocab, dtype=BF16, device=DEV)
    zd = flat.as_strided((3, vocab), (stride, 1))
    z = logits(gen(11), 3, vocab, BF16)
    zd.copy_(z)
    tok = torch.tensor([1, vocab // 2, 3])
    say("token_logprobs, rows 2^31 elements apart")
    p = rsx.token_logprobs(zd, tok.to(DEV), 4)
    ref, tol = so.token_logprobs(z, tok, 4)
    so.close(p.lse, ref["lse"], tol["lse"] + so.rounding(ref["lse"], F32))
    assert torch.equal(p.top_token.cpu(), ref["top_token"])
    rsx.token_logprobs_grad(zd, tok.to(DEV), p.lse, torch.ones(3, device=DEV), dlogits=zd)
    rz, tz = so.token_logprobs_grad(z, tok, p.lse.cpu(), None, torch.ones(3), None)
    so.close(zd, rz, tz + 1.01 * so.rounding(rz, BF16))


# --------------------------------------------- streams, graphs, refusals
def step_plans(seed):
    """Every operator on small inputs: (plans, the tensors they write)."""
    g = gen(seed)
    table, tok = rand(g, 300, 136).to(DEV), torch.randint(0, 300, (9000,), generator=g).to(DEV)
    e = rsx.Embedding(table, tok, scale=2.0)
    ck = rsx.Checkpoint((9000, 136), DEV)
    n = rsx.LayerNorm(e.out, checkpoint=ck)
    z = rand(g, 40, 9001, dtype=BF16).to(DEV)
    t2 = torch.randint(0, 9001, (40,), generator=g).to(DEV)
    lp = rsx.TokenLogprobs(z, t2, 5)
    lg = rsx.TokenLogprobsGrad(z, t2, lp.lse, torch.ones(40, device=DEV))
    ng = rsx.LayerNormGrad(n.out, ck, n.mean, n.rstd)
    grad = torch.empty_like(table)
    eg = rsx.EmbeddingGrad(ng.dx, tok, grad)
    un = rsx.CheckpointUnpack(ck)
    outs = [e.out, n.out, n.mean, n.rstd, lp.logprob, lp.entropy, lp.top_token, lg.dlogits, ng.dx, ng.dweight, ng.dbias, grad,
            un.out]
    return [e, n, lp, lg, ng, eg, un], outs


def test_other_stream_gives_the_same_bits():
    plans, outs = step_plans(1)
    for p in plans:
        p()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for p in plans:
        p(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(same_bits(a, b) for a, b in zip(want, outs))
    for o in outs:
        o.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for p in plans:
            p()
    s.synchronize()
    assert all(same_bits(a, b) for a, b in zip(want, outs))


def test_graph_replays_match_eager_calls():
    plans, outs = step_plans(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for p in plans:
            p()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in plans:
            p()
    for turn in range(4):
        plans[0].keep[0].mul_(1.5)  # another table
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        for p in plans:
            p()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, outs)), turn


def test_example_learns_and_its_ranks_agree():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, world = example.train(ranks=3, steps=30, vocab=200, dim=64, tokens=1000)
    # a model that knows nothing has ln 200 = 5.3; one that has learned the rule has little left
    assert 4.5 < losses[0] < 7.0 and losses[-1] < 2.0 and losses[-1] < losses[0]
    for r in world[1:]:
        assert all(same_bits(p, q) for p, q in zip(r.params, world[0].params))


def test_python_refusals():
    x = torch.zeros(4, 8, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    v = torch.zeros(4, device=DEV)
    bad = [
        lambda: rsx.Embedding(x, t.float()), lambda: rsx.Embedding(x, t[::2]), lambda: rsx.Embedding(x.int(), t),
        lambda: rsx.Embedding(x, t, out=torch.empty(4, 7, device=DEV)), lambda: rsx.Embedding(x.t(), t),
        lambda: rsx.Embedding(x[0], t), lambda: rsx.EmbeddingGrad(x, t[:3], x.clone()),
        lambda: rsx.EmbeddingGrad(x, t, x[:1].expand(4, 8)), lambda: rsx.LayerNorm(x.double()),
        lambda: rsx.LayerNorm(x, weight=v), lambda: rsx.LayerNorm(x, weight=torch.zeros(8, device=DEV, dtype=BF16)),
        lambda: rsx.LayerNorm(x, out=x.bfloat16()), lambda: rsx.LayerNorm(x, checkpoint=rsx.Checkpoint((4, 9), DEV)),
        lambda: rsx.LayerNorm(x[:, ::2]), lambda: rsx.LayerNorm(torch.zeros(2, 3, 8, device=DEV).transpose(0, 1)),
        lambda: rsx.LayerNorm(x.bfloat16(), torch.ones(8, device=DEV), torch.ones(8, device=DEV, dtype=BF16)),
        lambda: rsx.LayerNormGrad(x, x.bfloat16(), v, v), lambda: rsx.LayerNormGrad(x, x, v[:3], v),
        lambda: rsx.LayerNormGrad(x, rsx.Checkpoint((4, 9), DEV), v, v), lambda: rsx.CheckpointPack(x.int()),
        lambda: rsx.CheckpointUnpack(rsx.Checkpoint((4, 8), DEV), x.int()),
        lambda: rsx.TokenLogprobs(x, t, top=9), lambda: rsx.TokenLogprobs(x, t, top=-1), lambda: rsx.TokenLogprobs(x, t[:2]),
        lambda: rsx.TokenLogprobs(x[:, :0], t), lambda: rsx.TokenLogprobsGrad(x, t, v, v, None, v),
        lambda: rsx.TokenLogprobsGrad(x, t, v.double(), v), lambda: rsx.TokenLogprobsGrad(x, t, v, v[:1].expand(4)),
    ]
    for i, make in enumerate(bad):
        with pytest.raises(ValueError):
            make()
            say("not refused:", i)
    with pytest.raises(TypeError):
        rsx.LayerNorm(x, checkpoint=x)
    with pytest.raises(rsx.RsxError) as e:  # the row before is this one's output
        rsx.layer_norm(x.view(-1)[:24].view(3, 8), out=x.view(-1)[8:32].view(3, 8))
    assert e.value.status == 5
    # halves of one matrix interleave and do not overlap
    both = torch.randn(5, 16, device=DEV)
    want = rsx.layer_norm(both[:, :8].contiguous())[0]
    rsx.layer_norm(both[:, :8], out=both[:, 8:])
    assert torch.equal(both[:, 8:], want)
