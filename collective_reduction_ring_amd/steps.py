"""The operators of a training step that make the gradients the collectives reduce.

Embedding lookup and its gradient, layer norm and its gradients, 8-bit
checkpoints of activations, and token log probabilities with theirs
(include/rsx.h has the formulas).  As with the collectives, a class is a
prepared call over fixed tensors: making one checks every argument and
allocates what was not given (outputs, workspace), calling it enqueues the
kernels on the current stream (or ``stream``) and returns at once.  Tensors
may be refilled between calls.  The functions of the same names in lower case
prepare, call once and return the outputs.

What a plan allocates belongs to the stream that is current when it is made: a
first call on another stream has to be ordered after that one, as for any tensor
made there.  A plan has one workspace, so its calls are not for two streams at
once.  The functions with ``stream`` make their outputs and workspaces on that
stream; inputs have to be ready there.

Matrices are tensors whose last dimension is the row; the leading ones have to
fold into one row stride, so a column slice of a wider matrix is fine.  Rows
that are only read may be expanded (stride 0).  Nothing here records autograd
history: forward and backward are calls of their own.
"""
from __future__ import annotations

import math

import torch

from . import _lib as L

FLOATS = {torch.float32: L.RSX_FLOAT32, torch.bfloat16: L.RSX_BFLOAT16, torch.float16: L.RSX_FLOAT16}
TOKENS = {torch.int32: L.RSX_INT32, torch.int64: L.RSX_INT64}


def _tensor(t, what: str, device=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} is not a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} is not on a GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    return t


def _rows(t, what: str, types=FLOATS, device=None, shape=None, dtype=None, output: bool = False):
    """(rows, dim, row stride, type code) of a matrix."""
    _tensor(t, what, device)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if t.dtype not in types:
        raise ValueError(f"{what} has dtype {t.dtype}; one of {sorted(str(d) for d in types)}")
    if t.dim() < 1:
        raise ValueError(f"{what} needs at least one dimension")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    dim = t.shape[-1]
    rows = math.prod(t.shape[:-1])
    if t.numel() == 0 or t.is_contiguous():
        return rows, dim, dim, types[t.dtype]
    try:
        m = t.view(rows, dim)
    except RuntimeError:
        raise ValueError(f"{what}: the leading dimensions do not fold into rows of one stride") from None
    if dim > 1 and m.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row are not side by side")
    stride = m.stride(0) if rows > 1 else dim
    if stride < dim and not (stride == 0 and not output):
        raise ValueError(f"{what}: rows overlap")
    return rows, dim, stride, types[t.dtype]


def _vector(t, what: str, n: int, dtype, device):
    _tensor(t, what, device)
    if t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, expected {n}")
    if not t.is_contiguous():
        raise ValueError(f"{what} is not contiguous")
    return t


def _tokens(t, what: str, device, shape=None):
    _tensor(t, what, device)
    if t.dtype not in TOKENS:
        raise ValueError(f"{what} has dtype {t.dtype}; one of {sorted(str(d) for d in TOKENS)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} is not contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _first(first, vocab: int) -> int:
    first = int(first)
    if not -2 ** 63 <= first <= 2 ** 63 - max(vocab, 1):
        raise ValueError(f"first={first}: the ids of {vocab} rows from there leave 64 bits")
    return first


def _current_stream(index: int) -> int:
    # The handle alone: torch.cuda.current_stream() makes an object of it, which
    # took 2.7 of a small call's 6.4 us (this: 0.1).
    return torch._C._cuda_getCurrentRawStream(index)


def _as_stream(stream, device):
    """The stream object of a handle."""
    if not isinstance(stream, int):
        return stream
    # ExternalStream takes a handle of 0 for none, and makes a stream of its own.
    return torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)


def _ptr(t):
    return None if t is None else t.data_ptr()


class _Plan:
    """A prepared call: entry point, arguments, and the tensors they point to."""

    def _prepare(self, name: str, device, args, tensors) -> None:
        self.name, self.device = name, device
        self.fn = getattr(L.lib(), name)
        # ctypes values: a call converts none of them again
        self.args = tuple(typ(v) for typ, v in zip(self.fn.argtypes, args))
        self.keep = [t for t in tensors if t is not None]
        self.index = device.index
        self.home = _current_stream(self.index)

    def _workspace(self, nbytes: int, device):
        """(pointer, bytes) of a 256-byte aligned workspace, and the tensor that holds it."""
        if nbytes == 0:
            return None, 0, None
        t = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        return t.data_ptr() + (-t.data_ptr()) % 256, nbytes, t

    def __call__(self, stream=None) -> None:
        if torch.cuda.current_device() != self.index:
            with torch.cuda.device(self.device):
                return self(stream)
        if stream is None:
            handle = _current_stream(self.index)
        elif isinstance(stream, int):
            handle = stream
        else:
            handle = stream.cuda_stream
        st = self.fn(*self.args, handle)
        if st:
            L.check(self.name, st)
        if handle != self.home:
            self._use_on(stream, handle)

    def _use_on(self, stream, handle: int) -> None:
        # Memory freed after this call may be given out again on the stream it
        # was allocated on: the allocator has to know of this one's work.
        stream = torch.cuda.current_stream() if stream is None else _as_stream(stream, self.device)
        for t in self.keep:
            t.record_stream(stream)


def _once(tensor, stream, make) -> _Plan:
    """The plan that ``make`` gives, called on ``stream``; ``tensor`` is on its device."""
    device = getattr(tensor, "device", None)
    if stream is None or device is None or device.type != "cuda":  # the latter two are refused
        plan = make()
        plan(stream)
        return plan
    # Memory from the current stream's pool may have its last user still to run
    # there: outputs and workspace come from the pool of the stream that writes
    # them.  Either stream's work holds on to all of it.
    home = torch.cuda.current_stream(device)
    stream = _as_stream(stream, device)
    with torch.cuda.stream(stream):
        plan = make()
        plan(stream)
    for t in plan.keep:
        t.record_stream(stream)
        t.record_stream(home)
    return plan


class Embedding(_Plan):
    """Prepared lookup ``out[i] = scale * table[tokens[i] - first]``; a token
    outside the table gives a row of zeros.  ``out`` has the tokens' shape plus
    the table's row, in any of the float types (default: the table's).

    ``first`` is the token id of the table's first row: with the table cut by
    rows over W ranks, the sum all-reduce of the ranks' outputs is the lookup in
    the whole table."""

    def __init__(self, table, tokens, out=None, scale: float = 1.0, first: int = 0):
        _tensor(table, "table")
        dev = table.device
        if table.dim() != 2:
            raise ValueError("table needs two dimensions")
        vocab, dim, ts, tt = _rows(table, "table")
        _tokens(tokens, "tokens", dev)
        shape = (*tokens.shape, dim)
        if out is None:
            out = torch.empty(shape, dtype=table.dtype, device=dev)
        _, _, os_, ot = _rows(out, "out", device=dev, shape=shape, output=True)
        self.out = out
        self._prepare("rsx_embedding", dev, (_ptr(table), ts, vocab, dim, tt, _ptr(tokens), tokens.numel(),
                                             TOKENS[tokens.dtype], _first(first, vocab), float(scale), _ptr(out), os_, ot),
                      (table, tokens, out))


class EmbeddingGrad(_Plan):
    """Prepared gradient of the lookup in its table: ``grad[v] = (grad[v] if
    accumulate else 0) + scale * (sum of dout[i] over tokens[i] - first == v)``.
    Rows are summed in fp32, in parts and in the order of their positions (many
    tokens are sorted for it): the same bits on every run."""

    def __init__(self, dout, tokens, grad, scale: float = 1.0, first: int = 0, accumulate: bool = False):
        _tensor(grad, "grad")
        dev = grad.device
        if grad.dim() != 2:
            raise ValueError("grad needs two dimensions")
        vocab, dim, gs, gt = _rows(grad, "grad", output=True)
        _tokens(tokens, "tokens", dev)
        _, _, ds, dt = _rows(dout, "dout", device=dev, shape=(*tokens.shape, dim))
        n = tokens.numel()
        ws, wb, self._ws = self._workspace(L.lib().rsx_embedding_grad_workspace_size(n, vocab, dim), dev)
        self.grad = grad
        self._prepare("rsx_embedding_grad", dev, (_ptr(dout), ds, dt, _ptr(tokens), n, TOKENS[tokens.dtype],
                                                  _first(first, vocab), float(scale), _ptr(grad), gs, vocab, dim, gt,
                                                  int(bool(accumulate)), ws, wb),
                      (dout, tokens, grad, self._ws))


class Checkpoint:
    """An activation kept in 8 bits: int8 ``codes`` of the tensor's shape and one
    power-of-two ``scales`` byte for each 32 elements of a row, 33/32 bytes an
    element in all.  An element comes back within 1/64 of its block's largest
    magnitude (half of that but for the few codes the format clamps); a block
    with an infinity or a NaN comes back as NaN."""

    def __init__(self, shape, device="cuda"):
        self.shape = torch.Size(shape)
        if len(self.shape) < 1:
            raise ValueError("a checkpoint needs at least one dimension")
        self.dim = self.shape[-1]
        self.rows = math.prod(self.shape[:-1])
        blocks = -(-self.dim // L.RSX_CHECKPOINT_BLOCK)
        self.codes = torch.empty(self.shape, dtype=torch.int8, device=device)
        self.scales = torch.empty((*self.shape[:-1], blocks), dtype=torch.uint8, device=device)
        self.device = self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _checkpoint(c, what: str, shape, device) -> Checkpoint:
    if not isinstance(c, Checkpoint):
        raise TypeError(f"{what} is not a Checkpoint")
    if c.device != device:
        raise ValueError(f"{what} is on {c.device}, expected {device}")
    if tuple(c.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(c.shape)}, expected {tuple(shape)}")
    return c


class CheckpointPack(_Plan):
    """Prepared ``checkpoint = 8 bits of x``."""

    def __init__(self, x, checkpoint: Checkpoint | None = None):
        rows, dim, xs, xt = _rows(x, "x")
        c = Checkpoint(x.shape, x.device) if checkpoint is None else _checkpoint(checkpoint, "checkpoint", x.shape, x.device)
        self.checkpoint = c
        self._prepare("rsx_checkpoint_pack", x.device, (_ptr(x), xs, _ptr(c.codes), _ptr(c.scales), rows, dim, xt),
                      (x, c.codes, c.scales))


class CheckpointUnpack(_Plan):
    """Prepared ``out = the values that a checkpoint stands for``."""

    def __init__(self, checkpoint: Checkpoint, out=None, dtype=None):
        if not isinstance(checkpoint, Checkpoint):
            raise TypeError("checkpoint is not a Checkpoint")
        c = checkpoint
        if out is None:
            out = torch.empty(c.shape, dtype=torch.float32 if dtype is None else dtype, device=c.device)
        rows, dim, os_, ot = _rows(out, "out", device=c.device, shape=c.shape, dtype=dtype, output=True)
        self.out = out
        self._prepare("rsx_checkpoint_unpack", c.device, (_ptr(c.codes), _ptr(c.scales), _ptr(out), os_, rows, dim, ot),
                      (c.codes, c.scales, out))


def _weights(x, dim, **named):
    """The type code and dtype that the given weights share (x's type without any)."""
    dtype = None
    for what, w in named.items():
        if w is None:
            continue
        _tensor(w, what, x.device)
        if w.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"{what} has dtype {w.dtype}, expected {x.dtype} or torch.float32")
        if dtype is not None and w.dtype != dtype:
            raise ValueError(f"{what} has dtype {w.dtype}, expected {dtype} as the other weights")
        dtype = w.dtype
        _vector(w, what, dim, dtype, x.device)
    dtype = x.dtype if dtype is None else dtype
    return FLOATS[dtype], dtype


class LayerNorm(_Plan):
    """Prepared layer norm over the last dimension: ``out = (x - mean) * rstd *
    weight + bias``.  ``weight`` and ``bias`` are of x's type or float32, or
    None; ``out`` (x itself for in place) is of x's type; ``mean`` and ``rstd``
    (float32, a value per row) are what the gradient needs.  With a
    ``checkpoint`` the pass also keeps x in 8 bits there."""

    def __init__(self, x, weight=None, bias=None, out=None, eps: float = 1e-5, checkpoint: Checkpoint | None = None):
        rows, dim, xs, xt = _rows(x, "x")
        wt, _ = _weights(x, dim, weight=weight, bias=bias)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, _, os_, _ = _rows(out, "out", device=x.device, shape=x.shape, dtype=x.dtype, output=True)
        c = checkpoint
        if c is not None:
            _checkpoint(c, "checkpoint", x.shape, x.device)
        self.out, self.checkpoint = out, c
        # Rows without elements have no mean, and the call nothing to write.
        new = torch.empty if dim else lambda *a, **kw: torch.full(*a, math.nan, **kw)
        self.mean = new(x.shape[:-1], dtype=torch.float32, device=x.device)
        self.rstd = new(x.shape[:-1], dtype=torch.float32, device=x.device)
        codes, scales = (None, None) if c is None else (c.codes, c.scales)
        self._prepare("rsx_layer_norm", x.device,
                      (_ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(out), os_, _ptr(self.mean), _ptr(self.rstd),
                       _ptr(codes), _ptr(scales), rows, dim, float(eps), xt, wt),
                      (x, weight, bias, out, self.mean, self.rstd, codes, scales))


class LayerNormGrad(_Plan):
    """Prepared gradients of the layer norm: ``dx`` (of dout's type; dout or x
    itself for in place), ``dweight`` and ``dbias`` (of the weight's type,
    None with ``weights=False``).  ``x`` is the forward pass's input or a
    ``Checkpoint`` of it, ``mean`` and ``rstd`` its results."""

    def __init__(self, dout, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, weights: bool = True):
        rows, dim, ds, dt = _rows(dout, "dout")
        dev = dout.device
        packed = isinstance(x, Checkpoint)
        if packed:
            _checkpoint(x, "x", dout.shape, dev)
            xs, xp, codes, scales = dim, None, x.codes, x.scales
        else:
            _, _, xs, _ = _rows(x, "x", device=dev, shape=dout.shape, dtype=dout.dtype)
            xp, codes, scales = x, None, None
            if x.numel() == 0:  # no rows: an empty tensor has no address, and none is read
                xp = None
        _vector(mean, "mean", rows, torch.float32, dev)
        _vector(rstd, "rstd", rows, torch.float32, dev)
        wt, wdtype = _weights(dout, dim, weight=weight, dweight=dweight, dbias=dbias)
        if weights:
            dweight = torch.empty(dim, dtype=wdtype, device=dev) if dweight is None else dweight
            dbias = torch.empty(dim, dtype=wdtype, device=dev) if dbias is None else dbias
        if dx is None:
            dx = torch.empty(dout.shape, dtype=dout.dtype, device=dev)
        _, _, dxs, _ = _rows(dx, "dx", device=dev, shape=dout.shape, dtype=dout.dtype, output=True)
        ws, wb, self._ws = self._workspace(L.lib().rsx_layer_norm_grad_workspace_size(rows, dim), dev)
        self.dx, self.dweight, self.dbias = dx, dweight, dbias
        self._prepare("rsx_layer_norm_grad", dev,
                      (_ptr(dout), ds, _ptr(xp), xs, _ptr(codes), _ptr(scales), _ptr(mean), _ptr(rstd), _ptr(weight),
                       _ptr(dx), dxs, _ptr(dweight), _ptr(dbias), rows, dim, dt, wt, ws, wb),
                      (dout, xp, codes, scales, mean, rstd, weight, dx, dweight, dbias, self._ws))


class TokenLogprobs(_Plan):
    """Prepared log probabilities: for each row of ``logits`` the ``logprob`` of
    its token (0 for a token outside the row, as padding has), the ``entropy``,
    ``lse`` with ``lse_rest`` (what its rounding took: the gradient needs it for
    large logits), and with ``top`` > 0 the ``top`` largest logits' ``top_token``
    and ``top_logprob``, equal ones by the lower index.  A logit of -inf is masked."""

    def __init__(self, logits, tokens, top: int = 0):
        rows, vocab, zs, zt = _rows(logits, "logits")
        dev, lead = logits.device, logits.shape[:-1]
        _tokens(tokens, "tokens", dev, lead)
        if vocab == 0:
            raise ValueError("logits has empty rows")
        if not 0 <= top <= min(vocab, L.RSX_TOP_MAX):
            raise ValueError(f"top={top} outside [0, {min(vocab, L.RSX_TOP_MAX)}]")
        new = lambda *s: torch.empty((*lead, *s), dtype=torch.float32, device=dev)  # noqa: E731
        self.logprob, self.entropy, self.lse, self.lse_rest = new(), new(), new(), new()
        self.top_logprob = new(top) if top else None
        self.top_token = torch.empty((*lead, top), dtype=torch.int32, device=dev) if top else None
        ws, wb, self._ws = self._workspace(L.lib().rsx_token_logprobs_workspace_size(rows, vocab, top), dev)
        self._prepare("rsx_token_logprobs_rest", dev,
                      (_ptr(logits), zs, zt, _ptr(tokens), TOKENS[tokens.dtype], rows, vocab, top, _ptr(self.logprob),
                       _ptr(self.entropy), _ptr(self.lse), _ptr(self.lse_rest), _ptr(self.top_logprob), _ptr(self.top_token),
                       ws, wb),
                      (logits, tokens, self.logprob, self.entropy, self.lse, self.lse_rest, self.top_logprob, self.top_token,
                       self._ws))


class TokenLogprobsGrad(_Plan):
    """Prepared gradient in the logits for gradients ``dlogprob`` and (with
    ``entropy``) ``dentropy``; ``dlogits`` may be ``logits`` itself.  ``lse_rest``
    is the forward pass's: without it the probabilities are off by the rounding
    of ``lse``, 2^-24 of its size."""

    def __init__(self, logits, tokens, lse, dlogprob, entropy=None, dentropy=None, dlogits=None, lse_rest=None):
        rows, vocab, zs, zt = _rows(logits, "logits")
        dev = logits.device
        _tokens(tokens, "tokens", dev, logits.shape[:-1])
        if vocab == 0:
            raise ValueError("logits has empty rows")
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
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        _, _, ds, _ = _rows(dlogits, "dlogits", device=dev, shape=logits.shape, dtype=logits.dtype, output=True)
        self.dlogits = dlogits
        self._prepare("rsx_token_logprobs_grad_rest", dev,
                      (_ptr(logits), zs, zt, _ptr(tokens), TOKENS[tokens.dtype], _ptr(lse), _ptr(lse_rest), _ptr(entropy),
                       _ptr(dlogprob), _ptr(dentropy), _ptr(dlogits), ds, rows, vocab),
                      (logits, tokens, lse, lse_rest, entropy, dlogprob, dentropy, dlogits))


def embedding(table, tokens, out=None, scale: float = 1.0, first: int = 0, stream=None):
    """The rows of ``table`` that ``tokens`` name, scaled; see ``Embedding``."""
    return _once(table, stream, lambda: Embedding(table, tokens, out, scale, first)).out


def embedding_grad(dout, tokens, grad, scale: float = 1.0, first: int = 0, accumulate: bool = False, stream=None):
    """The table's gradient, into ``grad``; see ``EmbeddingGrad``."""
    return _once(grad, stream, lambda: EmbeddingGrad(dout, tokens, grad, scale, first, accumulate)).grad


def layer_norm(x, weight=None, bias=None, out=None, eps: float = 1e-5, checkpoint: Checkpoint | None = None, stream=None):
    """(out, mean, rstd) of a layer norm; see ``LayerNorm``."""
    p = _once(x, stream, lambda: LayerNorm(x, weight, bias, out, eps, checkpoint))
    return p.out, p.mean, p.rstd


def layer_norm_grad(dout, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, weights: bool = True, stream=None):
    """(dx, dweight, dbias) of a layer norm; see ``LayerNormGrad``."""
    p = _once(dout, stream, lambda: LayerNormGrad(dout, x, mean, rstd, weight, dx, dweight, dbias, weights))
    return p.dx, p.dweight, p.dbias


def checkpoint_pack(x, checkpoint: Checkpoint | None = None, stream=None) -> Checkpoint:
    """x in 8 bits; see ``Checkpoint``."""
    return _once(x, stream, lambda: CheckpointPack(x, checkpoint)).checkpoint


def checkpoint_unpack(checkpoint: Checkpoint, out=None, dtype=None, stream=None):
    """The values of a checkpoint, float32 unless ``out`` or ``dtype`` says otherwise."""
    return _once(checkpoint, stream, lambda: CheckpointUnpack(checkpoint, out, dtype)).out


def token_logprobs(logits, tokens, top: int = 0, stream=None) -> TokenLogprobs:
    """One pass over ``logits``; returns the plan, whose fields hold the results."""
    return _once(logits, stream, lambda: TokenLogprobs(logits, tokens, top))


def token_logprobs_grad(logits, tokens, lse, dlogprob, entropy=None, dentropy=None, dlogits=None, stream=None, lse_rest=None):
    """The gradient in the logits; see ``TokenLogprobsGrad``."""
    return _once(logits, stream, lambda: TokenLogprobsGrad(logits, tokens, lse, dlogprob, entropy, dentropy, dlogits,
                                                           lse_rest)).dlogits
