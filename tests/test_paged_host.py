"""Refusals of the paged-cache calls: everything here is decided on the host
before a launch (addresses are fake and never touched), so it needs no GPU."""

import ctypes

import numpy as np
import pytest

import rotate_then_quantize_b200 as rq
from rotate_then_quantize_b200 import binding as b

import paged

FAKE = 1 << 40
INV, UNS, MIS = b.SRFTQ_ERR_INVALID_ARG, b.SRFTQ_ERR_UNSUPPORTED, b.SRFTQ_ERR_MISALIGNED


def _at(i):
    return FAKE + (i << 34)


@pytest.fixture(scope="module")
def lib():
    return rq.load_library()


def _tables(lib, **kw):
    a = dict(n_seq=4, cached=_at(0), new=_at(1), page=16, free=_at(2), n_free=9, table=_at(3),
             max_pages=8, slots=_at(4), n_slots=10, lens=_at(5), starts=_at(6), counts=_at(7))
    a.update(kw)
    return lib.srftq_block_tables(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(n_seq=-1), INV), (dict(n_free=-1), INV), (dict(max_pages=-2), INV),
    (dict(n_slots=-1), INV), (dict(page=0), UNS), (dict(page=65537), UNS),
    (dict(n_seq=1 << 31), UNS), (dict(cached=None), INV), (dict(new=None), INV),
    (dict(free=None), INV), (dict(table=None), INV), (dict(slots=None), INV),
    (dict(lens=None), INV), (dict(starts=None), INV), (dict(counts=None), INV),
    (dict(cached=_at(0) + 2), MIS), (dict(slots=_at(4) + 4), MIS), (dict(counts=_at(7) + 1), MIS),
    (dict(lens=_at(0)), INV),                     # output over an input
    (dict(slots=_at(3) + 32), INV),               # two outputs over one another
])
def test_block_tables_refusals(lib, kw, want):
    assert _tables(lib, **kw) == want


def _quantize(lib, desc=(128, 2, 16, 4, 0), **kw):
    a = dict(S=2, N=8, x=_at(0), xs=8, signs=_at(1), lam=_at(2), slots=_at(3), codes=_at(4),
             scales=_at(5), rows=64)
    a.update(kw)
    d = rq.SrftqDesc(*desc) if desc else None
    return lib.srftq_quantize_paged(ctypes.byref(d) if d else None, *a.values(), None)


def _dequantize(lib, desc=(128, 2, 16, 4, 0), **kw):
    a = dict(S=2, N=8, codes=_at(4), scales=_at(5), rows=64, slots=_at(3), signs=_at(1),
             lam=_at(2), x=_at(0), xs=8)
    a.update(kw)
    d = rq.SrftqDesc(*desc) if desc else None
    return lib.srftq_dequantize_paged(ctypes.byref(d) if d else None, *a.values(), None)


@pytest.mark.parametrize("call", [_quantize, _dequantize])
@pytest.mark.parametrize("kw,want", [
    (dict(desc=None), INV), (dict(desc=(32, 2, 16, 4, 0)), UNS), (dict(desc=(128, 2, 8, 4, 0)), UNS),
    (dict(desc=(128, 2, 16, 5, 0)), UNS), (dict(desc=(128, 0, 16, 4, 0)), INV),
    (dict(desc=(128, 2, 16, 4, 2)), UNS), (dict(S=-1), INV), (dict(N=-1), INV),
    (dict(rows=-1), INV), (dict(N=1 << 31, xs=1 << 31), UNS), (dict(xs=7), INV),
    (dict(x=None), INV), (dict(slots=None), INV), (dict(codes=None), INV), (dict(scales=None), INV),
    (dict(signs=None), INV), (dict(lam=None), INV), (dict(x=_at(0) + 8), MIS),
    (dict(slots=_at(3) + 4), MIS), (dict(codes=_at(4) + 8), MIS),
    (dict(codes=_at(0)), INV), (dict(slots=_at(0)), None),
])
def test_paged_codec_refusals(lib, call, kw, want):
    if want is None:   # the slots may not lie in what the call writes
        want = INV
        kw = dict(slots=_at(4) if call is _quantize else _at(0))
    assert call(lib, **kw) == want


@pytest.mark.parametrize("call", [_quantize, _dequantize])
@pytest.mark.parametrize("kw", [dict(N=0), dict(S=0), dict(rows=0)])
def test_paged_codec_empty_calls(lib, call, kw):
    assert call(lib, **kw) == b.SRFTQ_OK


def _attention(lib, desc=(128, 2, 16, 4, 0), **kw):
    a = dict(dtype=0, n_seq=3, g=4, q=_at(0), kc=_at(1), ks=_at(2), ksg=_at(3), kl=_at(4),
             vc=_at(5), vs=_at(6), vsg=_at(7), vl=_at(8), pages=16, page=32, ptab=_at(9),
             prefix=100, table=_at(10), max_pages=8, lens=_at(11), scale=0.1, out=_at(12),
             lse=None, ws=_at(13), ws_bytes=1 << 30)
    a.update(kw)
    d = rq.SrftqDesc(*desc) if desc else None
    return lib.srftq_prefix_attention(ctypes.byref(d) if d else None, *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(desc=None), INV), (dict(desc=(32, 2, 16, 4, 0)), UNS), (dict(desc=(128, 2, 8, 4, 0)), UNS),
    (dict(dtype=2), UNS), (dict(n_seq=-1), INV), (dict(g=0), INV), (dict(g=17), UNS),
    (dict(prefix=-1), INV), (dict(prefix=1 << 31), UNS), (dict(pages=-1), INV),
    (dict(max_pages=-1), INV), (dict(page=0), UNS), (dict(page=1 << 17), UNS),
    (dict(max_pages=1 << 28), UNS), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(ptab=None), INV), (dict(table=None), INV),
    (dict(lens=None), INV), (dict(q=None), INV), (dict(kc=None), INV), (dict(vs=None), INV),
    (dict(out=None), INV), (dict(ws=None), INV), (dict(ws_bytes=64), INV),
    (dict(q=_at(0) + 2), MIS), (dict(ws=_at(13) + 8), MIS), (dict(lens=_at(11) + 2), MIS),
    (dict(lse=_at(14) + 2), MIS), (dict(out=_at(0)), INV), (dict(out=_at(5)), INV),
    (dict(lse=_at(12)), INV), (dict(ws=_at(10)), INV),
])
def test_prefix_attention_refusals(lib, kw, want):
    assert _attention(lib, **kw) == want


def test_prefix_attention_without_sequences(lib):
    assert _attention(lib, n_seq=0) == b.SRFTQ_OK


def test_workspace_sizes(lib):
    desc = rq.make_desc(128, 8, 16, 4)
    small = rq.srftq_prefix_attention_workspace(desc, 4, 1, 0)
    large = rq.srftq_prefix_attention_workspace(desc, 64, 8, 4096)
    assert 0 < small < large
    for bad in ((-1, 1, 0), (1, 0, 0), (1, 17, 0), (1, 1, -5)):
        with pytest.raises(rq.SrftqError):
            rq.srftq_prefix_attention_workspace(desc, *bad)


def test_python_refuses_host_tensors():
    import torch
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rq.srftq_block_tables(i, i, i, i.view(2, 2), 16, i.long(), i, i, i)
    h = torch.zeros((1, 4, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        rq.quantize_paged(h, h, h, i.long(), h, h)
    with pytest.raises(ValueError):
        rq.prefix_attention(h[0], h[0], h[0], h, h, h[0], h[0], h, h, i, i,
                            workspace=torch.zeros(1))


def test_plain_tables_by_hand():
    """The plain loop itself, on a case worked by hand: pages of 4, sequence 0
    holds 3 and gets 2 (its page has room for one), 1 is idle, 2 is new."""
    table = np.array([[7, -1], [5, -1], [-1, -1]], np.int32)
    t, slots, lens, starts, counts = paged.block_tables([3, 2, 0], [2, 0, 5], 4, [9, 1, 4, 6],
                                                        table, 9)
    assert t.tolist() == [[7, 9], [5, -1], [1, 4]]
    assert slots.tolist() == [31, 36, 4, 5, 6, 7, 16, -1, -1]
    assert (lens, starts, counts) == ([5, 2, 5], [0, 2, 2, 7], [3, 3, 7])


def test_plain_attention_by_hand():
    """One head, two pages of two rows, a prefix of one token: equal scores
    average the values; no token gives zeros."""
    k = np.zeros((4, 1, 2))
    v = np.arange(8.0).reshape(4, 1, 2)
    out, lse = paged.attention(np.ones((2, 1, 2)), k, v, np.array([[0, 1], [0, 1]]), [3, 0],
                               np.array([1]), 1, 2, 1.0)
    # tokens: prefix -> row 2; token 1 -> row 1; token 2 -> row 2 (page 1)
    np.testing.assert_allclose(out[0, 0], (v[2, 0] + v[1, 0] + v[2, 0]) / 3)
    assert lse[0, 0] == pytest.approx(np.log(3)) and lse[1, 0] == -np.inf
    assert (out[1] == 0).all()
