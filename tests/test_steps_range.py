"""The training-step operators without a GPU: further refusals, and what a plan does before its call."""
import contextlib

import pytest
import torch

from collective_reduction_ring_amd import _lib as L, steps
from test_abi import fake_ptrs
from test_steps import A, BAD, ALIAS, F32, I64, OK, call


def rest(z=A(1), tokens=A(2), rows=4, vocab=64, top=4, lp=A(3), ent=A(4), lse=A(5), lse_rest=A(8), tl=A(6), tt=A(7)):
    return call("rsx_token_logprobs_rest", z, vocab, F32, tokens, I64, rows, vocab, top, lp, ent, lse, lse_rest, tl, tt, None, 0)


def grad_rest(z=A(1), tokens=A(2), lse=A(3), lse_rest=A(8), ent=A(4), g=A(5), h=A(6), dz=A(7), rows=4, vocab=64):
    return call("rsx_token_logprobs_grad_rest", z, vocab, F32, tokens, I64, lse, lse_rest, ent, g, h, dz, vocab, rows, vocab)


@fake_ptrs
@pytest.mark.parametrize("fn,kw,want", [(rest, dict(lse_rest=A(8) + 2), BAD), (rest, dict(lse_rest=A(5) + 4), ALIAS),
                                        (rest, dict(lse_rest=A(1)), ALIAS), (rest, dict(vocab=0), BAD), (rest, dict(rows=0), OK),
                                        (grad_rest, dict(lse_rest=A(8) + 1), BAD), (grad_rest, dict(lse_rest=A(7) + 64), ALIAS),
                                        (grad_rest, dict(rows=0), OK), (grad_rest, dict(vocab=0), BAD)],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_refusals_of_the_forms_that_keep_the_rest(fn, kw, want):
    assert fn(**kw) == want


# ---- streams, with stand-ins for them, for tensors and for plans
class FakeTensor:
    device = torch.device("cuda:0")

    def __init__(self):
        self.recorded = []

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.mark.parametrize("handle", [0, 77])
def test_a_handle_of_0_is_the_default_stream(handle, monkeypatch):
    """A plan's memory is held for the stream of the call, not for one that 0 would make anew."""
    default, other = object(), object()
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: other)
    plan = steps._Plan()
    plan.device, plan.keep = FakeTensor.device, [FakeTensor()]
    plan._use_on(handle, handle)
    assert plan.keep[0].recorded == [default if handle == 0 else other]


class FakePlan:
    """Notes the stream that is current when it is made, and the one that it is called on."""

    def __init__(self, *args, **kw):
        self.made_on, self.called_on = FakePlan.current, None
        self.keep = [FakePlan.mine]
        self.out = self.grad = self.mean = self.rstd = self.dx = self.dweight = self.dbias = self.checkpoint = self.dlogits = None
        FakePlan.plans.append(self)

    def __call__(self, stream=None):
        self.called_on = stream


FUNCTIONS = {"embedding": ("Embedding", 2), "embedding_grad": ("EmbeddingGrad", 3), "layer_norm": ("LayerNorm", 1),
             "layer_norm_grad": ("LayerNormGrad", 4), "checkpoint_pack": ("CheckpointPack", 1),
             "checkpoint_unpack": ("CheckpointUnpack", 1), "token_logprobs": ("TokenLogprobs", 2),
             "token_logprobs_grad": ("TokenLogprobsGrad", 4)}


@pytest.mark.parametrize("given", ["object", "handle", "default"])
@pytest.mark.parametrize("name", FUNCTIONS)
def test_a_functions_memory_is_of_the_stream_it_runs_on(name, given, monkeypatch):
    """Outputs and workspace from another stream's pool could still be in use there."""
    class Stream:
        cuda_stream = 77

    home, default, wanted = object(), object(), Stream()

    @contextlib.contextmanager
    def use(s):
        FakePlan.current, before = s, FakePlan.current
        yield
        FakePlan.current = before

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: home)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: wanted if ptr == 77 else None)
    cls, n = FUNCTIONS[name]
    monkeypatch.setattr(steps, cls, FakePlan)
    FakePlan.current, FakePlan.plans, FakePlan.mine = home, [], FakeTensor()
    args = [FakeTensor() for _ in range(n)]
    stream, want = {"object": (wanted, wanted), "handle": (77, wanted), "default": (0, default)}[given]
    getattr(steps, name)(*args, stream=stream)
    p, = FakePlan.plans
    assert p.made_on is want and p.called_on is want
    assert want in p.keep[0].recorded and home in p.keep[0].recorded
    # without a stream, the current one: nothing to record
    FakePlan.plans, FakePlan.mine = [], FakeTensor()
    getattr(steps, name)(*args)
    p, = FakePlan.plans
    assert p.made_on is home and p.called_on is None and not p.keep[0].recorded


# ---- ids of a table's rows that 64 bits do not hold
def lookup(first, vocab=100):
    return call("rsx_embedding", A(1), 64, vocab, 64, F32, A(2), 0, I64, first, 1.0, A(3), 64, F32)


def lookup_grad(first, vocab=100):
    return call("rsx_embedding_grad", A(1), 64, F32, A(2), 0, I64, first, 1.0, A(3), 64, vocab, 64, F32, 0, None, 0)


@fake_ptrs
def test_rows_past_the_last_token_id_are_refused():
    """Their ids would wrap, and the smallest tokens name them."""
    most = 2 ** 63
    assert lookup(most - 100) == OK and lookup(-most) == OK
    assert lookup(most - 99) == BAD and lookup(most - 1, vocab=2) == BAD
    assert lookup_grad(most - 99) == BAD and lookup_grad(most - 1, vocab=2) == BAD
    assert lookup(most - 1, vocab=0) == OK and lookup_grad(most - 1, vocab=0) == OK


@pytest.mark.parametrize("first", [2 ** 64 + 5, 2 ** 63, 2 ** 63 - 3, -2 ** 63 - 1])
def test_python_refuses_firsts_beyond_64_bits(first):
    """ctypes cuts them to 64 bits without a word."""
    with pytest.raises(ValueError, match="first"):
        steps._first(first, 4)
    assert steps._first(2 ** 63 - 4, 4) == 2 ** 63 - 4 and steps._first(-2 ** 63, 4) == -2 ** 63
