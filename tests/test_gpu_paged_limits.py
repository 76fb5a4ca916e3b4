"""The shared-prefix attention at the longest positions that it takes: a small
pool whose two pages the tables name over and over, so that a token's weight is
its row's weight times the number of times its page is named.

Tolerance: that of paged.check_attention, 8 * 2^-11 of the row's root mean square
and half a step of the output, plus the accumulation: a part adds 16 tokens at a
time to float32 sums, and the matrix units may cut each sum off instead of
rounding it, one step of at most 2^-23 of it an addition."""

import math

import numpy as np
import pytest

import oracle
import rotate_then_quantize_b200 as rq

import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = 2 ** 31 - 65536
PAGE, D = 4096, 64


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _pool(rng, toward=None):
    """Two pages of quantised vectors, those of the second 12 further along
    `toward`: their scores for a query of length 8 that way are 12 higher."""
    x = rng.standard_normal((1, 2 * PAGE, 1, D))
    if toward is not None:
        x[:, PAGE:] += 12 * toward
    x = x.astype(np.float16)
    signs = np.where(rng.random((1, 1, D)) < 0.5, -1, 1).astype(np.int8)
    lam = oracle.calibrate_lambda(x, signs, 2 * PAGE, 0).astype(np.float32)
    z = oracle.quantize(x, signs, lam, 16, 4, 0)
    hat = oracle.dequantize(z["codes"], z["scales"], signs, lam, D, 16, 4, 0)["xhat64"]
    dev = (_t(z["codes"][0]), _t(z["scales"][0].view(np.float16)), _t(signs[0]), _t(lam[0]))
    return dev, hat[0, :, 0]


def _check(out, q, khat, vhat, count, adds):
    import torch
    s = q.double().cpu().numpy() @ khat.T / math.sqrt(D)
    p = np.exp(s - s.max(-1, keepdims=True)) * count
    ref = p @ vhat / p.sum(-1, keepdims=True)
    rms = np.sqrt((ref * ref).mean(-1, keepdims=True))
    tol = (torch.finfo(q.dtype).eps / 2 * np.abs(ref)
           + (8 * paged.U + adds * 2.0 ** -23) * np.maximum(np.abs(ref), rms))
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())


def _tokens(n, pages):
    """How often each row of the pool is among the first n tokens; the last three
    of `pages` are the second page, all others the first."""
    count = np.zeros(2 * PAGE)
    count[:PAGE] = pages - 3
    count[PAGE:] = 3
    count[2 * PAGE - (pages * PAGE - n):] -= 1     # the last page ends inside
    return count


def _queries(rng, n_seq, g, dtype):
    import torch
    u = rng.standard_normal(D)
    u /= np.linalg.norm(u)
    q = 8 * u + 0.3 * rng.standard_normal((n_seq, g, D))
    return u, _t(q).to(getattr(torch, dtype))


@pytest.mark.parametrize("dtype,g", [("bfloat16", 1), ("float16", 2)])
def test_own_tokens_up_to_the_limit(dtype, g):
    import torch
    rng = np.random.default_rng(g)
    u, q = _queries(rng, 3, g, dtype)
    (k, khat), (v, vhat) = _pool(rng, u), _pool(rng)
    pages = (MOST - 1) // PAGE
    table = torch.zeros((3, pages), dtype=torch.int32, device=DEV)
    table[0, -3:] = 1
    n = pages * PAGE - 7
    lens = torch.tensor([n, 9, 0], dtype=torch.int32, device=DEV)
    out = rq.prefix_attention(q, *k, *v, table, lens, page_size=PAGE)
    assert rq.srftq_check_device() == 0
    # one KV head: 1184 chunks, four warps each
    _check(out[0], q[0], khat, vhat, _tokens(n, pages), n / 1184 / 4 / 16)
    few = np.zeros(2 * PAGE)
    few[:9] = 1
    _check(out[1], q[1], khat, vhat, few, 1)
    assert (out[2] == 0).all()


@pytest.mark.parametrize("dtype,g", [("bfloat16", 1), ("bfloat16", 16), ("float16", 16)])
def test_prefix_up_to_the_limit(dtype, g):
    """By the warp-level kernel (two rows) and the tcgen05 one (32)."""
    import torch
    rng = np.random.default_rng(10 + g)
    u, q = _queries(rng, 2, g, dtype)
    (k, khat), (v, vhat) = _pool(rng, u), _pool(rng)
    n = MOST - 1
    pages = -(-n // PAGE)
    table = torch.zeros(pages, dtype=torch.int32, device=DEV)
    table[-3:] = 1
    lens = torch.tensor([n, 4000], dtype=torch.int32, device=DEV)
    out = rq.prefix_attention(q, *k, *v, torch.zeros((2, 1), dtype=torch.int32, device=DEV), lens,
                              table, n, page_size=PAGE)
    assert rq.srftq_check_device() == 0
    # at least 148 blocks of two units, or 592 of four warps
    _check(out[0], q[0], khat, vhat, _tokens(n, pages), n / (296 if g > 1 else 2368) / 16)
    few = np.zeros(2 * PAGE)
    few[:4000] = 1
    _check(out[1], q[1], khat, vhat, few, 250)
