"""The training-step operators without a GPU: refusals, sizes, and the oracle.

Calls with made-up addresses have to be refused before any HIP call; they are
skipped where a GPU is visible.
"""
import ctypes
import math

import pytest
import torch

import collective_reduction_ring_amd as rsx
from collective_reduction_ring_amd import _lib as L
import step_oracle as so
from test_abi import fake_ptrs

F32, BF16, I32, F16, I64, I8 = (L.RSX_FLOAT32, L.RSX_BFLOAT16, L.RSX_INT32, L.RSX_FLOAT16, L.RSX_INT64, L.RSX_INT8)
OK, BAD, TYPE, UNSUPPORTED, ALIAS = 0, 1, 2, 4, 5


def A(k):
    """Made-up device address number k, 1 GiB apart."""
    return 0x7f0000000000 + (k << 30)


def call(name, *args):
    return getattr(L.lib(), name)(*args, None)


def embedding(table=A(1), ts=64, vocab=100, dim=64, tt=F32, tokens=A(2), n=8, kt=I64, out=A(3), os=64, ot=F32):
    return call("rsx_embedding", table, ts, vocab, dim, tt, tokens, n, kt, 0, 1.0, out, os, ot)


def embedding_grad(dout=A(1), ds=64, dt=F32, tokens=A(2), n=8, kt=I64, grad=A(3), gs=64, vocab=100, dim=64, gt=F32, ws=A(4),
                   wb=1 << 20):
    return call("rsx_embedding_grad", dout, ds, dt, tokens, n, kt, 0, 1.0, grad, gs, vocab, dim, gt, 0, ws, wb)


def norm(x=A(1), xs=64, w=A(2), b=A(3), y=A(4), ys=64, mean=A(5), rstd=A(6), codes=A(7), scales=A(8), rows=4, dim=64, t=F32,
         wt=F32):
    return call("rsx_layer_norm", x, xs, w, b, y, ys, mean, rstd, codes, scales, rows, dim, 1e-5, t, wt)


def norm_grad(dy=A(1), dys=64, x=A(2), xs=64, codes=None, scales=None, mean=A(3), rstd=A(4), w=A(5), dx=A(6), dxs=64, dw=A(7),
              db=A(8), rows=4, dim=64, t=F32, wt=F32, ws=A(9), wb=1 << 20):
    return call("rsx_layer_norm_grad", dy, dys, x, xs, codes, scales, mean, rstd, w, dx, dxs, dw, db, rows, dim, t, wt, ws, wb)


def pack(x=A(1), xs=64, codes=A(2), scales=A(3), rows=4, dim=64, t=F32):
    return call("rsx_checkpoint_pack", x, xs, codes, scales, rows, dim, t)


def unpack(codes=A(2), scales=A(3), out=A(1), os=64, rows=4, dim=64, t=F32):
    return call("rsx_checkpoint_unpack", codes, scales, out, os, rows, dim, t)


def logprobs(z=A(1), zs=64, t=F32, tokens=A(2), kt=I64, rows=4, vocab=64, top=4, lp=A(3), ent=A(4), lse=A(5), tl=A(6), tt=A(7),
             ws=None, wb=0):
    return call("rsx_token_logprobs", z, zs, t, tokens, kt, rows, vocab, top, lp, ent, lse, tl, tt, ws, wb)


def logprobs_grad(z=A(1), zs=64, t=F32, tokens=A(2), kt=I64, lse=A(3), ent=A(4), g=A(5), h=A(6), dz=A(7), dzs=64, rows=4,
                  vocab=64):
    return call("rsx_token_logprobs_grad", z, zs, t, tokens, kt, lse, ent, g, h, dz, dzs, rows, vocab)


BIG = 1 << 31
REFUSALS = [
    (embedding, dict(tt=I32), TYPE), (embedding, dict(ot=I8), TYPE), (embedding, dict(kt=F32), TYPE),
    (embedding, dict(table=None), BAD), (embedding, dict(out=None), BAD), (embedding, dict(tokens=None), BAD),
    (embedding, dict(table=A(1) + 2), BAD), (embedding, dict(tokens=A(2) + 4), BAD), (embedding, dict(out=A(3) + 1, ot=BF16), BAD),
    (embedding, dict(ts=63), BAD), (embedding, dict(os=63), BAD), (embedding, dict(os=0), BAD),
    (embedding, dict(vocab=BIG), UNSUPPORTED), (embedding, dict(dim=BIG, ts=BIG, os=BIG), UNSUPPORTED),
    (embedding, dict(n=BIG), UNSUPPORTED), (embedding, dict(ts=1 << 44), UNSUPPORTED), (embedding, dict(ts=1 << 62), UNSUPPORTED),
    (embedding, dict(out=A(1)), ALIAS), (embedding, dict(out=A(2)), ALIAS),
    (embedding, dict(out=A(1) + 32 * 4, os=128, ts=128, dim=64), ALIAS),
    (embedding_grad, dict(dt=I32), TYPE), (embedding_grad, dict(gt=I64), TYPE), (embedding_grad, dict(kt=I8), TYPE),
    (embedding_grad, dict(dout=None), BAD), (embedding_grad, dict(grad=None), BAD), (embedding_grad, dict(gs=32), BAD),
    (embedding_grad, dict(ds=32), BAD), (embedding_grad, dict(ws=None), BAD), (embedding_grad, dict(ws=A(4) + 128), BAD),
    (embedding_grad, dict(wb=255), BAD), (embedding_grad, dict(grad=A(1)), ALIAS), (embedding_grad, dict(grad=A(4)), ALIAS),
    (embedding_grad, dict(ws=A(2)), ALIAS), (embedding_grad, dict(n=BIG), UNSUPPORTED),
    (norm, dict(t=I32), TYPE), (norm, dict(t=BF16, wt=F16), TYPE), (norm, dict(wt=BF16), TYPE),
    (norm, dict(x=None), BAD), (norm, dict(y=None), BAD), (norm, dict(codes=None), BAD), (norm, dict(scales=None), BAD),
    (norm, dict(xs=32), BAD), (norm, dict(ys=32), BAD), (norm, dict(w=A(2) + 2), BAD), (norm, dict(mean=A(5) + 1), BAD),
    (norm, dict(y=A(1) + 4), ALIAS), (norm, dict(y=A(1), ys=128), ALIAS), (norm, dict(y=A(2)), ALIAS),
    (norm, dict(rstd=A(5)), ALIAS), (norm, dict(codes=A(4)), ALIAS), (norm, dict(scales=A(7) + 8), ALIAS),
    (norm, dict(rows=BIG), UNSUPPORTED), (norm, dict(dim=BIG), UNSUPPORTED),
    (norm_grad, dict(t=I8), TYPE), (norm_grad, dict(wt=F16), TYPE), (norm_grad, dict(dy=None), BAD),
    (norm_grad, dict(x=None), BAD), (norm_grad, dict(x=None, codes=A(10)), BAD), (norm_grad, dict(codes=A(10), scales=A(11)), BAD),
    (norm_grad, dict(mean=None), BAD), (norm_grad, dict(rstd=None), BAD), (norm_grad, dict(dx=None), BAD),
    (norm_grad, dict(ws=None), BAD), (norm_grad, dict(wb=64), BAD), (norm_grad, dict(dx=A(1) + 4), ALIAS),
    (norm_grad, dict(dx=A(2), dxs=128), ALIAS), (norm_grad, dict(dw=A(8)), ALIAS), (norm_grad, dict(dw=A(5)), ALIAS),
    (norm_grad, dict(ws=A(6)), ALIAS), (norm_grad, dict(rows=BIG), UNSUPPORTED),
    (pack, dict(t=I32), TYPE), (pack, dict(x=None), BAD), (pack, dict(codes=None), BAD), (pack, dict(xs=8), BAD),
    (pack, dict(codes=A(1)), ALIAS), (pack, dict(scales=A(2)), ALIAS), (pack, dict(rows=BIG), UNSUPPORTED),
    (unpack, dict(t=I8), TYPE), (unpack, dict(out=None), BAD), (unpack, dict(os=0), BAD), (unpack, dict(out=A(2)), ALIAS),
    (unpack, dict(dim=BIG), UNSUPPORTED),
    (logprobs, dict(t=I32), TYPE), (logprobs, dict(kt=F32), TYPE), (logprobs, dict(z=None), BAD), (logprobs, dict(lp=None), BAD),
    (logprobs, dict(lse=None), BAD), (logprobs, dict(tl=None), BAD), (logprobs, dict(tt=None), BAD), (logprobs, dict(vocab=0), BAD),
    (logprobs, dict(top=65), BAD), (logprobs, dict(top=-1), BAD), (logprobs, dict(vocab=3, zs=3), BAD), (logprobs, dict(zs=8), BAD),
    (logprobs, dict(vocab=1 << 17, zs=1 << 17), BAD),  # such rows are cut into slices and need a workspace
    (logprobs, dict(lp=A(1)), ALIAS), (logprobs, dict(lse=A(3)), ALIAS), (logprobs, dict(tl=A(7)), ALIAS),
    (logprobs, dict(vocab=BIG, zs=BIG), UNSUPPORTED),
    (logprobs_grad, dict(t=I64), TYPE), (logprobs_grad, dict(kt=BF16), TYPE), (logprobs_grad, dict(dz=None), BAD),
    (logprobs_grad, dict(ent=None), BAD), (logprobs_grad, dict(lse=None), BAD), (logprobs_grad, dict(g=None), BAD),
    (logprobs_grad, dict(vocab=0), BAD), (logprobs_grad, dict(dzs=8), BAD), (logprobs_grad, dict(dz=A(1) + 4), ALIAS),
    (logprobs_grad, dict(dz=A(1), dzs=128), ALIAS), (logprobs_grad, dict(dz=A(5)), ALIAS),
    (logprobs_grad, dict(rows=BIG), UNSUPPORTED),
]


@fake_ptrs
@pytest.mark.parametrize("fn,kw,want", REFUSALS, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_refusals(fn, kw, want):
    assert fn(**kw) == want


@fake_ptrs
@pytest.mark.parametrize("fn,kw", [(embedding, dict(n=0)), (embedding, dict(dim=0)), (embedding_grad, dict(vocab=0)),
                                   (embedding_grad, dict(dim=0)), (norm, dict(rows=0)), (norm, dict(dim=0)),
                                   (norm_grad, dict(dim=0)), (pack, dict(rows=0)), (unpack, dict(dim=0)),
                                   (logprobs, dict(rows=0)), (logprobs_grad, dict(rows=0))],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_nothing_to_do(fn, kw):
    assert fn(**kw) == OK


def test_workspace_sizes():
    lib = L.lib()
    assert lib.rsx_embedding_grad_workspace_size(0, 100, 64) == 0
    assert lib.rsx_embedding_grad_workspace_size(BIG, 100, 64) == 0
    # keys and positions twice, and two partial rows of fp32 for each chunk of 128
    n, d = 65536, 4096
    need = lib.rsx_embedding_grad_workspace_size(n, 50000, d)
    assert 16 * n + 2 * (n // 128) * d * 4 <= need <= 16 * n + 2 * (n // 128) * d * 4 + (1 << 20)
    assert lib.rsx_layer_norm_grad_workspace_size(0, 64) == 0
    assert lib.rsx_layer_norm_grad_workspace_size(1, 64) == 2 * 64 * 4
    assert lib.rsx_token_logprobs_workspace_size(4096, 1000, 4) == 0
    assert lib.rsx_token_logprobs_workspace_size(1, 1 << 17, 4) > 0
    assert lib.rsx_token_logprobs_workspace_size(1, 1 << 17, 65) == 0


def test_python_refuses_host_tensors():
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for make in (lambda: rsx.Embedding(x, t), lambda: rsx.EmbeddingGrad(x, t, x), lambda: rsx.LayerNorm(x),
                 lambda: rsx.LayerNormGrad(x, x, x, x), lambda: rsx.CheckpointPack(x),
                 lambda: rsx.TokenLogprobs(x, t), lambda: rsx.TokenLogprobsGrad(x, t, x, x)):
        with pytest.raises(ValueError, match="not on a GPU"):
            make()
    with pytest.raises(TypeError):
        rsx.LayerNorm([1.0])
    with pytest.raises(TypeError):
        rsx.CheckpointUnpack(x)


def test_header_constants():
    from test_abi import _header_int
    assert _header_int("RSX_TOP_MAX") == L.RSX_TOP_MAX
    assert _header_int("RSX_CHECKPOINT_BLOCK") == L.RSX_CHECKPOINT_BLOCK == so.BLOCK


# ---- the oracle against differences and against torch in 64 bits
def _differences(f, x, h=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        lo, hi = x.clone().reshape(-1), x.clone().reshape(-1)
        lo[i] -= h
        hi[i] += h
        g.reshape(-1)[i] = (f(hi.view_as(x)) - f(lo.view_as(x))) / (2 * h)
    return g


def test_oracle_norm_gradient_is_the_difference():
    g = torch.Generator().manual_seed(1)
    x, w, b, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 7), (7,), (7,), (3, 7)))
    f = lambda x, w, b: (so.layer_norm(x, w, b, 1e-5)[0][0] * dy).sum()  # noqa: E731
    _, mean, rstd = so.layer_norm(x, w, b, 1e-5)[0]
    dx, dw, db = so.layer_norm_grad(dy, x, mean, rstd, w)[0]
    # differences of step 1e-5 in 64 bits: about 1e-10 of the step's square, 1e-11 of rounding
    assert (dx - _differences(lambda v: f(v, w, b), x)).abs().max() < 1e-7
    assert (dw - _differences(lambda v: f(x, v, b), w)).abs().max() < 1e-7
    assert (db - _differences(lambda v: f(x, w, v), b)).abs().max() < 1e-7


def test_oracle_logprob_gradient_is_the_difference():
    g = torch.Generator().manual_seed(2)
    z = torch.randn(3, 9, generator=g, dtype=torch.float64)
    tok = torch.tensor([4, -1, 8])
    gl, gh = torch.randn(3, generator=g, dtype=torch.float64), torch.randn(3, generator=g, dtype=torch.float64)

    def f(z):
        o = so.token_logprobs(z, tok, 0)[0]
        return (o["logprob"] * gl + o["entropy"] * gh).sum()
    o = so.token_logprobs(z, tok, 3)[0]
    dz, _ = so.token_logprobs_grad(z, tok, o["lse"], o["entropy"], gl, gh)
    assert (dz - _differences(f, z)).abs().max() < 1e-7
    assert torch.equal(o["top_token"].long(), torch.topk(z, 3).indices)
    logp = torch.log_softmax(z, 1)
    assert (o["top_logprob"] - torch.topk(logp, 3).values).abs().max() < 1e-12
    assert (o["entropy"] + (logp.exp() * logp).sum(1)).abs().max() < 1e-12


def test_oracle_checkpoint_format():
    x = torch.tensor([[1.0, -1.984375, 0.5, 0.0078125, 0.0078126, 2.0 ** -7 * 1.5, 0.0]])
    codes, scales = so.checkpoint(x)
    # 2^0 <= 1.98 < 2^1: steps of 2^-6; half a step rounds to even
    assert scales.tolist() == [[121]]
    assert codes.tolist() == [[64, -127, 32, 0, 1, 1, 0]]
    codes, scales = so.checkpoint(torch.tensor([[1.999, 0.0], [math.inf, 1.0], [0.0, 0.0]]))
    assert codes.tolist() == [[127, 0], [0, 0], [0, 0]] and scales.tolist() == [[121], [255], [0]]
    assert torch.isnan(so.checkpoint_values(codes, scales)[1]).all()
