"""The step's matrix products at the ends of their ranges, without a GPU.

Calls with made-up addresses have to be refused before any HIP call.
"""
import pytest

import product_digits as pd
from test_abi import fake_ptrs
from test_products import ortho
from test_steps import A, ALIAS, BAD, BF16, F32, UNSUPPORTED

TALL = (1 << 21) + 1


@fake_ptrs
@pytest.mark.parametrize("kw", [
    # (rows - 1) * stride is 0 in 64 bits: the span of a matrix looked like that of one row
    dict(xs=1 << 43), dict(os=1 << 43), dict(xs=1 << 43, os=1 << 43), dict(xs=1 << 44, os=1 << 44, t=BF16),
    dict(xs=1 << 43, rows=(1 << 21) + 3), dict(os=1 << 43, batch=2, xm=TALL * 64, om=64), dict(xs=1 << 43, batch=2, xm=64, om=TALL * 64),
    # and where nothing wraps, spans past 2^45 bytes
    dict(xs=1 << 25), dict(os=1 << 25)], ids=str)
def test_update_strides_whose_span_leaves_the_range(kw):
    args = dict(rows=TALL, cols=64, xs=64, os=64, xm=0, om=0, batch=1, t=F32, out=A(100), ws=A(200), wb=1 << 40)
    assert ortho(**{**args, **kw}) == UNSUPPORTED


HIP = 6  # everything was accepted, and there is no GPU


@fake_ptrs
@pytest.mark.parametrize("kw,want", [
    # three matrices side by side in rows of 192 or more
    (dict(xs=192, xm=64), HIP), (dict(os=192, om=64), HIP), (dict(xs=200, xm=66, os=192, om=64), HIP),
    (dict(xs=192, xm=64, os=192, om=64, out=A(1)), HIP),
    # rows that meet: the last matrix's with the first one's next, or a matrix's with the next one's
    (dict(xs=191, xm=64), BAD), (dict(os=191, om=64), BAD), (dict(xs=192, xm=63), BAD), (dict(os=192, om=63), BAD),
    # an output behind the input's columns, on them, and between its matrices (which is not looked at so closely)
    (dict(xs=400, xm=64, os=400, om=64, out=A(1) + 192 * 2), HIP), (dict(xs=400, xm=64, os=400, om=64, out=A(1) + 190 * 2), ALIAS),
    (dict(xs=400, xm=128, os=400, om=128, out=A(1) + 64 * 2), ALIAS), (dict(xs=192, xm=64, ws=A(1)), ALIAS)], ids=str)
def test_update_of_interleaved_stacks(kw, want):
    args = dict(batch=3, rows=100, cols=64, xm=6400, om=6400)
    assert ortho(**{**args, **kw}) == want


def test_the_digits_bounds_find_a_lost_part():
    """The bounds that the GPU's fp32 products have to meet pass six products of parts, and not five of them."""
    for rows, dim, hidden, names in pd.BLOCKS:
        if rows * dim * hidden >= 1 << 27:  # (of the others' shape, and long to multiply here)
            continue
        inputs = pd.block_inputs(rows, dim, hidden, names)
        ref, bound = pd.block(*inputs, names), pd.block_bounds(rows, dim, hidden)
        for lost in [None] + pd.SEGMENTS[1:] if rows * dim * hidden < 1 << 23 else [None, (2, 0)]:
            got = pd.block(*inputs, names, [s for s in pd.SEGMENTS if s != lost])
            for n in names:
                assert (pd.off(got[n], ref[n]) > bound[n]) == (lost is not None), (rows, dim, hidden, n, lost)
    for rows, vocab, dim, n in pd.HEADS:
        if rows * vocab * dim >= 1 << 27:
            continue
        inputs = pd.head_inputs(rows, vocab, dim, n)
        ref, bound = pd.head(*inputs, n), pd.head_bounds(rows, vocab, dim)[n]
        for lost in [None] + pd.SEGMENTS[1:] if rows * vocab * dim < 1 << 23 else [None, (2, 0)]:
            got = pd.head(*inputs, n, [s for s in pd.SEGMENTS if s != lost])
            assert (pd.head_off(n, got, ref) > bound) == (lost is not None), (rows, vocab, dim, n, lost)
