"""The training-step operators without a GPU: further refusals, and what a plan does before its call."""
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


# ---- streams, with stand-ins for them and for tensors
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
