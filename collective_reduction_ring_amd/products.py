"""The matrix products of a training step that its framework would otherwise make
of several: the gated feed-forward block and its gradients, log probabilities
from the hidden state without logits, and the update orthogonalised after the
gradients' all-reduce (include/rsx.h has the formulas).

Classes are plans, functions one call, and streams, workspaces and matrices are
as in ``steps``.  A matrix of 16-bit elements whose address, row stride or width
is no multiple of 16 bytes is copied in every call.
"""
from __future__ import annotations

import math

import torch

from . import _lib as L
from .steps import FLOATS, TOKENS, _once, _Plan, _ptr, _rows, _tensor, _tokens, _vector

ACTIVATIONS = {"silu": L.RSX_ACT_SILU, "gelu": L.RSX_ACT_GELU, "gelu_tanh": L.RSX_ACT_GELU_TANH, "relu": L.RSX_ACT_RELU}


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation={name!r}: one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def _copies(*matrices) -> int:
    """Whether the library copies one of the (tensor, rows, width, stride) before it multiplies."""
    for t, rows, width, stride in matrices:
        if rows and width and t.element_size() == 2 and (
                t.data_ptr() % 16 or width % 8 or (rows > 1 and (stride % 8 or stride < width or stride >= 1 << 22))):
            return 1
    return 0


def _matrix(t, what: str, rows: int, dim: int, like, output: bool = False, dtype=None):
    """Row stride of a two-dimensional matrix of the given shape."""
    _tensor(t, what, like.device)
    return _rows(t, what, device=like.device, shape=(rows, dim), dtype=like.dtype if dtype is None else dtype, output=output)[2]


def _gradient_type(like, **named):
    """The dtype that the given weight gradients share: the matrices' or float32."""
    dtype = None
    for what, t in named.items():
        if t is None:
            continue
        _tensor(t, what, like.device)
        if t.dtype not in (like.dtype, torch.float32):
            raise ValueError(f"{what} has dtype {t.dtype}, expected {like.dtype} or torch.float32")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype} as the others")
        dtype = t.dtype
    return like.dtype if dtype is None else dtype


def _block(x, w_gate, w_up, w_down):
    """(rows, dim, hidden, type, strides of x and the three matrices)."""
    rows, dim, xs, xt = _rows(x, "x")
    _tensor(w_gate, "w_gate", x.device)
    if w_gate.dim() != 2:
        raise ValueError("w_gate needs two dimensions")
    hidden = w_gate.shape[0]
    return rows, dim, hidden, xt, (xs, _matrix(w_gate, "w_gate", hidden, dim, x), _matrix(w_up, "w_up", hidden, dim, x),
                                   _matrix(w_down, "w_down", dim, hidden, x))


class FeedForward(_Plan):
    """Prepared gated feed-forward block: ``out = (act(x @ w_gate.T) * (x @ w_up.T))
    @ w_down.T``, with ``w_gate`` and ``w_up`` of (hidden, dim), ``w_down`` of (dim,
    hidden), all of x's type, and ``activation`` "silu", "gelu", "gelu_tanh" or
    "relu".  With ``keep`` the two projections stay in ``gate`` and ``up`` (float32)
    for the gradient."""

    def __init__(self, x, w_gate, w_up, w_down, out=None, activation: str = "silu", keep: bool = False):
        rows, dim, hidden, xt, (xs, gs, us, ds) = _block(x, w_gate, w_up, w_down)
        act = _activation(activation)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        os_ = _rows(out, "out", device=x.device, shape=x.shape, dtype=x.dtype, output=True)[2]
        self.out, self.gate, self.up = out, None, None
        if keep:
            self.gate, self.up = (torch.empty((*x.shape[:-1], hidden), dtype=torch.float32, device=x.device) for _ in range(2))
        copies = _copies((x, rows, dim, xs), (w_gate, hidden, dim, gs), (w_up, hidden, dim, us), (w_down, dim, hidden, ds))
        ws, wb, self._ws = self._workspace(L.lib().rsx_feed_forward_workspace_size(rows, dim, hidden, xt, copies), x.device)
        # Tensors without elements have no address, and the library takes no half of a pair.
        kept = (self.gate, self.up) if keep and rows and hidden else (None, None)
        self._prepare("rsx_feed_forward", x.device,
                      (_ptr(x), xs, _ptr(w_gate), gs, _ptr(w_up), us, _ptr(w_down), ds, _ptr(out), os_, _ptr(kept[0]), _ptr(kept[1]),
                       rows, dim, hidden, act, xt, ws, wb),
                      (x, w_gate, w_up, w_down, out, self.gate, self.up, self._ws))


class FeedForwardGrad(_Plan):
    """Prepared gradients of the block from the ``gate`` and ``up`` that it kept:
    ``dx`` (None with ``inputs=False``) of x's type, and ``dw_gate``, ``dw_up`` and
    ``dw_down`` (None with ``weights=False``), all three of x's type or float32,
    added to what they hold with ``accumulate``."""

    def __init__(self, dout, x, w_gate, w_up, w_down, gate, up, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                 activation: str = "silu", accumulate: bool = False, inputs: bool = True, weights: bool = True):
        rows, dim, hidden, xt, (xs, gs, us, ds) = _block(x, w_gate, w_up, w_down)
        dev, act = x.device, _activation(activation)
        ys = _rows(dout, "dout", device=dev, shape=x.shape, dtype=x.dtype)[2]
        _vector(gate, "gate", rows * hidden, torch.float32, dev)
        _vector(up, "up", rows * hidden, torch.float32, dev)
        given = [t is not None for t in (dw_gate, dw_up, dw_down)]
        if accumulate and weights and not all(given):
            raise ValueError("accumulate needs dw_gate, dw_up and dw_down")
        wtype = _gradient_type(x, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down)
        shapes = {"dw_gate": (hidden, dim), "dw_up": (hidden, dim), "dw_down": (dim, hidden)}
        grads, strides = [], []
        for (what, shape), t in zip(shapes.items(), (dw_gate, dw_up, dw_down)):
            if weights:
                t = torch.empty(shape, dtype=wtype, device=dev) if t is None else t
                strides.append(_matrix(t, what, *shape, x, output=True, dtype=wtype))
            else:
                t = None
                strides.append(0)
            grads.append(t)
        dxs = 0
        if inputs:
            dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if dx is None else dx
            dxs = _rows(dx, "dx", device=dev, shape=x.shape, dtype=x.dtype, output=True)[2]
        else:
            dx = None
        self.dx, (self.dw_gate, self.dw_up, self.dw_down) = dx, grads
        copies = _copies((dout, rows, dim, ys), (x, rows, dim, xs), (w_gate, hidden, dim, gs), (w_up, hidden, dim, us),
                         (w_down, dim, hidden, ds))
        ws, wb, self._ws = self._workspace(L.lib().rsx_feed_forward_grad_workspace_size(rows, dim, hidden, xt, copies), dev)
        self._prepare("rsx_feed_forward_grad", dev,
                      (_ptr(dout), ys, _ptr(x), xs, _ptr(w_gate), gs, _ptr(w_up), us, _ptr(w_down), ds, _ptr(gate), _ptr(up),
                       _ptr(dx), dxs, _ptr(grads[0]), strides[0], _ptr(grads[1]), strides[1], _ptr(grads[2]), strides[2],
                       rows, dim, hidden, act, xt, FLOATS[wtype], int(bool(accumulate)), ws, wb),
                      (dout, x, w_gate, w_up, w_down, gate, up, dx, *grads, self._ws))


def _head(hidden, weight, tokens, scale):
    """(rows, vocab, dim, type, strides of hidden and weight, scale)."""
    rows, dim, hs, ht = _rows(hidden, "hidden")
    _tensor(weight, "weight", hidden.device)
    if weight.dim() != 2:
        raise ValueError("weight needs two dimensions")
    vocab = weight.shape[0]
    if vocab == 0:
        raise ValueError("weight has no rows")
    ws = _matrix(weight, "weight", vocab, dim, hidden)
    _tokens(tokens, "tokens", hidden.device, hidden.shape[:-1])
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError(f"scale={scale} is not finite")
    return rows, vocab, dim, ht, hs, ws, scale


class LinearLogprobs(_Plan):
    """Prepared ``TokenLogprobs`` of the logits ``scale * hidden @ weight.T``, which
    are never in memory: ``logprob``, ``entropy``, ``lse`` and ``lse_rest`` of each
    row of ``hidden``, with ``weight`` of (vocab, dim)."""

    def __init__(self, hidden, weight, tokens, scale: float = 1.0):
        rows, vocab, dim, ht, hs, wst, scale = _head(hidden, weight, tokens, scale)
        dev = hidden.device
        new = lambda: torch.empty(hidden.shape[:-1], dtype=torch.float32, device=dev)  # noqa: E731
        self.logprob, self.entropy, self.lse, self.lse_rest = new(), new(), new(), new()
        copies = _copies((hidden, rows, dim, hs), (weight, vocab, dim, wst))
        ws, wb, self._ws = self._workspace(L.lib().rsx_linear_logprobs_workspace_size(rows, vocab, dim, ht, copies), dev)
        self._prepare("rsx_linear_logprobs", dev,
                      (_ptr(hidden), hs, _ptr(weight), wst, ht, _ptr(tokens), TOKENS[tokens.dtype], rows, vocab, dim, scale,
                       _ptr(self.logprob), _ptr(self.entropy), _ptr(self.lse), _ptr(self.lse_rest), ws, wb),
                      (hidden, weight, tokens, self.logprob, self.entropy, self.lse, self.lse_rest, self._ws))


class LinearLogprobsGrad(_Plan):
    """Prepared gradients of ``LinearLogprobs`` for gradients ``dlogprob`` and (with
    ``entropy``) ``dentropy``: ``dhidden`` of hidden's type, ``dweight`` of hidden's
    type or float32, added to what it holds with ``accumulate``; None with
    ``inputs=False`` or ``weights=False``.  A row without a gradient (padding, or
    masked out of the loss) adds nothing, whatever it holds.  The logits are multiplied again, a piece
    of the vocabulary at a time; ``lse`` and ``lse_rest`` are the forward pass's."""

    def __init__(self, hidden, weight, tokens, lse, dlogprob, entropy=None, dentropy=None, dhidden=None, dweight=None,
                 lse_rest=None, scale: float = 1.0, accumulate: bool = False, inputs: bool = True, weights: bool = True):
        rows, vocab, dim, ht, hs, wst, scale = _head(hidden, weight, tokens, scale)
        dev = hidden.device
        _vector(lse, "lse", rows, torch.float32, dev)
        _vector(dlogprob, "dlogprob", rows, torch.float32, dev)
        if lse_rest is not None:
            _vector(lse_rest, "lse_rest", rows, torch.float32, dev)
        if dentropy is None:
            entropy = None
        else:
            if entropy is None:
                raise ValueError("dentropy needs entropy")
            _vector(entropy, "entropy", rows, torch.float32, dev)
            _vector(dentropy, "dentropy", rows, torch.float32, dev)
        if accumulate and weights and dweight is None:
            raise ValueError("accumulate needs dweight")
        wtype, dhs, dws = _gradient_type(hidden, dweight=dweight), 0, 0
        if inputs:
            dhidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=dev) if dhidden is None else dhidden
            dhs = _rows(dhidden, "dhidden", device=dev, shape=hidden.shape, dtype=hidden.dtype, output=True)[2]
        else:
            dhidden = None
        if weights:
            dweight = torch.empty((vocab, dim), dtype=wtype, device=dev) if dweight is None else dweight
            dws = _matrix(dweight, "dweight", vocab, dim, hidden, output=True, dtype=wtype)
        else:
            dweight = None
        self.dhidden, self.dweight = dhidden, dweight
        copies = _copies((hidden, rows, dim, hs), (weight, vocab, dim, wst))
        ws, wb, self._ws = self._workspace(L.lib().rsx_linear_logprobs_grad_workspace_size(rows, vocab, dim, ht, copies), dev)
        self._prepare("rsx_linear_logprobs_grad", dev,
                      (_ptr(hidden), hs, _ptr(weight), wst, ht, _ptr(tokens), TOKENS[tokens.dtype], _ptr(lse), _ptr(lse_rest),
                       _ptr(entropy), _ptr(dlogprob), _ptr(dentropy), _ptr(dhidden), dhs, _ptr(dweight), dws, FLOATS[wtype],
                       int(bool(accumulate)), rows, vocab, dim, scale, ws, wb),
                      (hidden, weight, tokens, lse, lse_rest, entropy, dlogprob, dentropy, dhidden, dweight, self._ws))


def _stack(t, what: str, output: bool = False):
    """(batch, rows, cols, row stride, matrix stride) of a matrix or a stack of them."""
    _tensor(t, what)
    if t.dtype not in FLOATS:
        raise ValueError(f"{what} has dtype {t.dtype}; one of {sorted(str(d) for d in FLOATS)}")
    if t.dim() < 2:
        raise ValueError(f"{what} needs two dimensions or more")
    rows, cols = t.shape[-2:]
    batch = math.prod(t.shape[:-2])
    if t.numel() == 0 or t.is_contiguous():
        return batch, rows, cols, cols, rows * cols
    try:
        m = t.view(batch, rows, cols)
    except RuntimeError:
        raise ValueError(f"{what}: the leading dimensions do not fold into matrices of one stride") from None
    if cols > 1 and m.stride(2) != 1:
        raise ValueError(f"{what}: the elements of a row are not side by side")
    stride = m.stride(1) if rows > 1 else cols
    each = m.stride(0) if batch > 1 else (rows - 1) * stride + cols
    if stride < cols and not (stride == 0 and not output):
        raise ValueError(f"{what}: rows overlap")
    beside = each >= cols and (batch - 1) * each + cols <= stride  # side by side in rows of all of them
    if each < (rows - 1) * stride + cols and not beside and not (each == 0 and not output):
        raise ValueError(f"{what}: matrices overlap")
    return batch, rows, cols, stride, each


class NewtonSchulz(_Plan):
    """Prepared orthogonalisation of an update, or of each of a stack (..., rows,
    cols): ``out`` (``update`` itself for in place) is of its type and shape.
    ``steps`` times X = a X + (b A + c A A) X with A = X X^T, from ``update``
    divided by its Frobenius norm (plus ``eps``); the singular values all come
    near 1.  The matrices of a stack may lie side by side in their rows, as the
    slices of a fused projection do.  No value on the way may pass 16: none does
    with coefficients that keep the singular values near 1."""

    def __init__(self, update, out=None, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7):
        batch, rows, cols, us, um = _stack(update, "update")
        steps, eps = int(steps), float(eps)
        if steps < 1:
            raise ValueError(f"steps={steps}: at least 1")
        if not eps >= 0:
            raise ValueError(f"eps={eps} is negative")
        a, b, c = (float(v) for v in coefficients)
        if out is None:
            out = torch.empty(update.shape, dtype=update.dtype, device=update.device)
        _tensor(out, "out", update.device)
        if out.dtype != update.dtype:
            raise ValueError(f"out has dtype {out.dtype}, expected {update.dtype}")
        if out.shape != update.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(update.shape)}")
        _, _, _, os_, om = _stack(out, "out", output=True)
        self.out = out
        ws, wb, self._ws = self._workspace(L.lib().rsx_newton_schulz_workspace_size(batch, rows, cols), update.device)
        self._prepare("rsx_newton_schulz", update.device,
                      (_ptr(update), us, um, _ptr(out), os_, om, batch, rows, cols, steps, a, b, c, eps, FLOATS[update.dtype], ws, wb),
                      (update, out, self._ws))


def feed_forward(x, w_gate, w_up, w_down, out=None, activation: str = "silu", keep: bool = False, stream=None) -> FeedForward:
    """The gated feed-forward block; returns the plan, whose fields hold ``out`` and what it kept."""
    return _once(x, stream, lambda: FeedForward(x, w_gate, w_up, w_down, out, activation, keep))


def feed_forward_grad(dout, x, w_gate, w_up, w_down, gate, up, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                      activation: str = "silu", accumulate: bool = False, inputs: bool = True, weights: bool = True, stream=None):
    """(dx, dw_gate, dw_up, dw_down); see ``FeedForwardGrad``."""
    p = _once(x, stream, lambda: FeedForwardGrad(dout, x, w_gate, w_up, w_down, gate, up, dx, dw_gate, dw_up, dw_down, activation,
                                                 accumulate, inputs, weights))
    return p.dx, p.dw_gate, p.dw_up, p.dw_down


def linear_logprobs(hidden, weight, tokens, scale: float = 1.0, stream=None) -> LinearLogprobs:
    """Log probabilities from hidden states; returns the plan, whose fields hold the results."""
    return _once(hidden, stream, lambda: LinearLogprobs(hidden, weight, tokens, scale))


def linear_logprobs_grad(hidden, weight, tokens, lse, dlogprob, entropy=None, dentropy=None, dhidden=None, dweight=None, lse_rest=None,
                         scale: float = 1.0, accumulate: bool = False, inputs: bool = True, weights: bool = True, stream=None):
    """(dhidden, dweight); see ``LinearLogprobsGrad``."""
    p = _once(hidden, stream, lambda: LinearLogprobsGrad(hidden, weight, tokens, lse, dlogprob, entropy, dentropy, dhidden, dweight,
                                                         lse_rest, scale, accumulate, inputs, weights))
    return p.dhidden, p.dweight


def newton_schulz(update, out=None, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, stream=None):
    """The orthogonalised update; see ``NewtonSchulz``."""
    return _once(update, stream, lambda: NewtonSchulz(update, out, steps, coefficients, eps)).out
