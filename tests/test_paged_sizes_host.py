"""Sizes that the shared-prefix attention refuses are refused by the question for
its workspace too, which would not fit 64 bits for some of them."""

import ctypes

import pytest

import rotate_then_quantize_b200 as rq
from rotate_then_quantize_b200 import binding as b


def _workspace(heads, n_seq, g, prefix, d=256):
    desc = rq.SrftqDesc(d, heads, 16, 4, 0)
    return rq.load_library().srftq_prefix_attention_workspace(ctypes.byref(desc), n_seq, g, prefix)


@pytest.mark.parametrize("heads,n_seq,g,prefix", [
    (1 << 16, 1 << 15, 1, 0), ((1 << 20) - 1, (1 << 27) - 5000, 16, 1 << 30), (1 << 19, 1 << 26, 16, 0),
    (8, 1 << 26, 4, 5000)])
def test_more_query_heads_than_the_call_takes(heads, n_seq, g, prefix):
    assert n_seq * heads * g >= 1 << 31
    assert _workspace(heads, n_seq, g, prefix) == b.SRFTQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("heads,n_seq,g,prefix", [
    ((1 << 20) - 1, 128, 16, 1 << 30), (8, (1 << 27) - 5000, 1, (1 << 31) - 65537), (1, 1, 1, 0),
    (1 << 16, (1 << 15) - 1, 1, 12345)])
def test_the_most_that_it_takes(heads, n_seq, g, prefix):
    """A size above what the queries alone take, and one that grows with the batch."""
    assert n_seq * heads * g < 1 << 31
    size = _workspace(heads, n_seq, g, prefix)
    assert size >= n_seq * heads * g * 256 * 4
    assert n_seq == 1 or size > _workspace(heads, n_seq // 2, g, prefix)
