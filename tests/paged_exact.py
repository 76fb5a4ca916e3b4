"""What fp16 outputs of the shared-prefix attention are held to, and a numpy model
of the kernels' arithmetic for them.

With fp16 outputs the queries, keys and weights are held as an fp16 value and its
rest, 22 bits together, and the values sigma c as one fp16 number. So against a
reference that takes those fp16 values (and all else in 64 bits) the output is off
by its own rounding, eps / 2, and by what is left of float32:

* a score is a float32 sum of 3 d / 16 products (48 at d = 256), each of which may
  cut off one step, 2^-23 of the sum at most: 6e-6 of scores up to 5, 3e-5; the
  rests' own rounding is 2^-22, the offsets' (warp-level kernel) 2^-17 of a score's
  standard deviation, and ex2's 2^-22. Independent from token to token or nearly so,
  these move an output by less than 3e-5 of the row's root mean square, 4 standard
  deviations of which are 1.2e-4;
* a part's sums take 2 tokens / 16 additions, at most 2000 here in four or more
  parts: 500 * 2^-24 = 3e-5 of them.

Both are below TIGHT = 2^-13. A rest that is lost leaves 2^-11 / sqrt 6 = 2e-4 of
the root mean square (standard deviation), which 10^3 coordinates do not hide.

For queries five times as long (PEAKED) scores reach 30 and the sums' steps 2e-4,
and a row is a few tokens: 2^-11; a lost rest of keys or query is 2e-4 of a score of
standard deviation 6, 1.2e-3, times the difference of two values.
"""

import numpy as np

import oracle

import paged

TIGHT, PEAKED = 2.0 ** -13, 2.0 ** -11


def rounded_values(codes, scales, signs, lam, bits, group, rot):
    """The rows that fp16 values sigma c stand for, [rows, H, d] in 64 bits."""
    c = oracle.unpack_codes(codes, bits).astype(np.float64)
    s = np.asarray(scales).view(np.float16).astype(np.float64)
    v = (c * np.repeat(s, group, -1)).astype(np.float16).astype(np.float64)
    y = v * np.asarray(lam, np.float32).astype(np.float64)
    return oracle.unrotate(y[None], signs[None], rot)[0]


def worst(out, ref, slack):
    """Largest error over its bound, eps / 2 |ref| + slack max(|ref|, rms)."""
    rms = np.sqrt(np.mean(ref * ref, -1, keepdims=True))
    tol = 2.0 ** -11 * np.abs(ref) + slack * np.maximum(np.abs(ref), rms)
    assert (out[(rms == 0)[..., 0]] == 0).all()
    live = (rms > 0)[..., 0]
    return float((np.abs(out - ref)[live] / tol[live]).max(initial=0.0))


def _split(x, rest):
    hi = x.astype(np.float16).astype(np.float64)
    return hi + (x - hi).astype(np.float16).astype(np.float64) if rest else hi


def model(q, k, v, lam_k, lam_v, signs_k, signs_v, rot, lost=None):
    """fp16 outputs [rows, d] of queries q [rows, d] over tokens of one head as the
    kernels compute them, k and v the sigma c [tokens, d] in 64 bits; lost names a rest
    that is left out: "query", "keys" or "weights"."""
    d = q.shape[-1]
    z = oracle.rotate(q[None, :, None], signs_k[None, None], rot)[0, :, 0] * lam_k / np.sqrt(d)
    z = (z * np.log2(np.e)).astype(np.float32).astype(np.float64)
    e = 13 - np.floor(np.log2(np.abs(z).max(-1, keepdims=True)))
    z = _split(z * 2.0 ** e, lost != "query") * 2.0 ** -e
    x = (z @ _split(k, lost != "keys").T).astype(np.float32).astype(np.float64)
    p = np.exp2(x - x.max(-1, keepdims=True) + 7).astype(np.float32).astype(np.float64)
    acc = _split(p, lost != "weights") @ v.astype(np.float16).astype(np.float64)
    y = acc / p.sum(-1, keepdims=True) * lam_v
    out = oracle.unrotate(y[None, :, None], signs_v[None, None], rot)[0, :, 0]
    return out.astype(np.float16).astype(np.float64)
