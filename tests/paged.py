"""Plain statements of the paged-cache operators, for their tests (numpy, 64 bits).

Tolerances of the attention, fixed before any kernel ran. The codes and scales
are the same on both sides, so only roundings differ:

* the output is rounded once to its type: half a step, eps/2 relative;
* inside, the weights p, the values sigma c, the keys sigma c and the rotated
  query may each be held in fp16 (relative half step u = 2^-11, standard
  deviation at most u / sqrt 3). Each of the four moves an output coordinate by
  independent errors of the tokens: relative to the row's root mean square the
  weights and values by at most u / sqrt 3 each, keys and query by the score's
  error, u / sqrt 3 times the scores' standard deviation s (about 1 to 1.5 for
  the inputs here) each. Together sqrt(2 + 2 s^2) u / sqrt 3 <= 1.5 u; the
  largest of 10^5 such errors is below 5.5 of that, 8 u.

So: |out - ref| <= eps/2 |ref| + 8 * 2^-11 max(|ref|, rms of the row). The
log-sum-exp moves by the scores' errors, averaged: 8 u (absolute, in nats).
"""

from __future__ import annotations

import numpy as np

import oracle

U = 2.0 ** -11


def block_tables(cached, new, page, free, table, n_slots):
    """The step's table, slots, lengths, row starts and counts, by a plain loop."""
    table = table.copy()
    max_pages = table.shape[1]
    slots, lens, starts, taken = [], [], [0], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        first, last = -(-c // page), -(-(c + n) // page)
        for p in range(first, min(last, max_pages)):
            table[b, p] = free[taken] if taken < len(free) else -1
            taken += 1
        for t in range(c, c + n):
            p = t // page
            ok = p < max_pages and table[b, p] >= 0
            slots.append(int(table[b, p]) * page + t % page if ok else -1)
        lens.append(c + n)
        starts.append(len(slots))
    counts = [min(taken, len(free)), taken, len(slots)]
    slots = (slots + [-1] * n_slots)[:n_slots]
    return table, np.array(slots, np.int64), lens, starts, counts


def rows_of(table, tokens, page, n_pages):
    """Pool rows of the tokens, -1 where the table names no page."""
    p = np.asarray(table, np.int64)[tokens // page]
    return np.where((p >= 0) & (p < n_pages), p * page + tokens % page, -1)


def attention(q, khat, vhat, block_table, seq_lens, prefix_table, prefix_len, page, scale,
              spread=None):
    """(out, lse) in 64 bits; khat, vhat [rows, H, d] dequantised pools.

    spread, a [n_seq, HQ, 1] array, gets the standard deviation that the fp16
    roundings inside give a coordinate of each row, to first order. With e_t the
    error of score t and f_t, g_t the relative ones of weight and value, the
    output moves by sum_t p_t (e_t (v_t - out) + (f_t + g_t) v_t). The errors
    are independent; f, g have standard deviation u / sqrt 3 at most, e_t that
    times the root of scale^2 sum_j 2 (q_j k_tj)^2 (key and query), which in the
    rotated domain is 2 scale^2 |q|^2 |k_t|^2 / d, up to 1 + 2 cos^2(q, k_t) for
    a key along the query: 1.5 covers cosines up to 0.5. R is orthogonal, so a
    coordinate's share of the squared error is the row's over d."""
    n_seq, HQ, d = q.shape
    H = khat.shape[1]
    g = HQ // H
    n_pages = khat.shape[0] // page
    cap = max(prefix_len, block_table.shape[1] * page)
    out, lse = np.zeros((n_seq, HQ, d)), np.full((n_seq, HQ), -np.inf)
    for b in range(n_seq):
        n = min(max(int(seq_lens[b]), 0), cap)
        t = np.arange(n)
        rows = np.concatenate([
            rows_of(prefix_table, t[:prefix_len], page, n_pages) if prefix_len else t[:0],
            rows_of(block_table[b], t[prefix_len:], page, n_pages) if n > prefix_len else t[:0]])
        rows = rows[rows >= 0].astype(np.int64)
        if not rows.size:
            continue
        for hq in range(HQ):
            s = khat[rows, hq // g] @ np.asarray(q[b, hq], np.float64) * scale
            m = s.max()
            p = np.exp(s - m)
            lse[b, hq] = m + np.log(p.sum())
            v = vhat[rows, hq // g]
            out[b, hq] = p @ v / p.sum()
            if spread is not None:
                k = khat[rows, hq // g]
                qn = np.linalg.norm(np.asarray(q[b, hq], np.float64))
                e2 = 1.5 * 2 * (scale * qn) ** 2 * (k * k).sum(-1) / d
                part = e2 * ((v - out[b, hq]) ** 2).sum(-1) + 2 * (v * v).sum(-1)
                w2 = (p / p.sum()) ** 2
                spread[b, hq] = U / np.sqrt(3) * np.sqrt(w2 @ part / d)
    return out, lse


def check_attention(out, ref, eps):
    """The elementwise bound of the module's docstring; returns the worst ratio."""
    out = np.asarray(out, np.float64)
    assert np.isfinite(out).all()
    rms = np.sqrt(np.mean(ref * ref, -1, keepdims=True))
    tol = eps / 2 * np.abs(ref) + 8 * U * np.maximum(np.abs(ref), rms)
    empty = (rms == 0)[..., 0]
    assert (out[empty] == 0).all(), "a row without tokens is zero"
    ratio = np.abs(out - ref)[~empty] / tol[~empty]
    worst = float(ratio.max(initial=0.0))
    assert worst <= 1.0, worst
    return worst


def cache(rng, rows, H, d, bits, group, kind, spread=None):
    """Quantised random K or V pool: codes, scale bits, signs, lambda, and the
    dequantised rows in 64 bits."""
    x = rng.standard_normal((1, rows, H, d))
    if spread is not None:
        x = x * spread
    x = x.astype(np.float16)
    signs = np.where(rng.random((1, H, d)) < 0.5, -1, 1).astype(np.int8)
    lam = oracle.calibrate_lambda(x, signs, min(rows, 256), kind).astype(np.float32)
    z = oracle.quantize(x, signs, lam, group, bits, kind)
    hat = oracle.dequantize(z["codes"], z["scales"], signs, lam, d, group, bits, kind)["xhat64"]
    return z["codes"][0], z["scales"][0], signs[0], lam[0], hat[0]
