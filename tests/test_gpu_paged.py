"""GPU tests of the paged cache: block tables, the paged codec and the
shared-prefix attention, each against a plain statement in 64 bits."""

import math

import numpy as np
import pytest

import oracle
import rotate_then_quantize_b200 as rq

import paged
import parity

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------------------
# Block tables
# ---------------------------------------------------------------------------

def _tables_case(rng, n_seq, page, most_cached, most_new, short=0, narrow=0, idle=0.3):
    cached = rng.integers(0, most_cached + 1, n_seq)
    new = np.where(rng.random(n_seq) < idle, 0, rng.integers(0, most_new + 1, n_seq))
    held, total = -(-cached // page), -(-(cached + new) // page)
    width = max(int(total.max(initial=0)) + 1 - narrow, 1)
    n_pages = int(total.sum()) + 3
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((n_seq, width), -7, np.int32)   # -7: entries that stay as they are
    at = 0
    for b in range(n_seq):
        k = min(int(held[b]), width)
        table[b, :k] = ids[at:at + k]
        at += int(held[b])
    free = ids[at:]
    need = int(np.maximum(np.minimum(total, width) - held, 0).sum())
    free = free[:max(need - short, 0) if short else need + 2]
    return cached, new, table, free, int(new.sum())


@pytest.mark.parametrize("n_seq,page,cached,new,short,narrow,pad", [
    (1, 16, 0, 1, 0, 0, 0), (1, 1, 5, 3, 0, 0, 2), (32, 64, 1000, 1, 0, 0, 0),
    (33, 24, 100, 77, 0, 0, 9), (1023, 16, 40, 50, 0, 0, 1), (1025, 7, 9, 5, 0, 0, 0),
    (3000, 16, 64, 40, 0, 0, 5000), (3, 128, 5000, 9000, 0, 0, 3), (40, 16, 50, 60, 11, 0, 4),
    (40, 16, 50, 60, 10 ** 6, 0, 4), (40, 16, 50, 200, 0, 5, 4), (5, 65536, 100000, 70000, 0, 0, 1),
])
def test_block_tables(n_seq, page, cached, new, short, narrow, pad):
    rng = np.random.default_rng(n_seq * 7 + page + new + short + narrow)
    c, n, table, free, total = _tables_case(rng, n_seq, page, cached, new, short, narrow)
    want = paged.block_tables(c, n, page, free, table, total + pad)
    dev = _t(table)
    slots, lens, starts, counts = rq.block_tables(_t(c.astype(np.int32)), _t(n.astype(np.int32)),
                                                  _t(free), dev, page, total + pad)
    np.testing.assert_array_equal(dev.cpu().numpy(), want[0])
    np.testing.assert_array_equal(slots.cpu().numpy(), want[1])
    assert lens.tolist() == want[2] and starts.tolist() == want[3] and counts.tolist() == want[4]


def test_block_tables_odd_inputs():
    """No sequences, no slots, negative lengths, fewer slots than rows, and a
    table without columns."""
    import torch
    i32 = dict(dtype=torch.int32, device=DEV)
    none = torch.zeros(0, **i32)
    slots, lens, starts, counts = rq.block_tables(none, none, none, torch.zeros((0, 3), **i32), 16,
                                                  3)
    assert slots.tolist() == [-1] * 3 and starts.tolist() == [0] and counts.tolist() == [0] * 3
    table = torch.full((3, 2), -1, **i32)
    free = torch.tensor([4, 2, 9, 7], **i32)
    slots, lens, starts, counts = rq.block_tables(
        torch.tensor([-5, 0, 3], **i32), torch.tensor([2, -1, 4], **i32), free, table, 4, 3)
    assert lens.tolist() == [2, 0, 7] and starts.tolist() == [0, 2, 2, 6]
    # sequence 2's partly filled page is entry 0, which holds no page: no slot
    assert slots.tolist() == [16, 17, -1] and counts.tolist() == [2, 2, 6]
    assert table.tolist() == [[4, -1], [-1, -1], [-1, 2]]
    slots, _, _, counts = rq.block_tables(torch.tensor([0], **i32), torch.tensor([2], **i32), free,
                                          torch.zeros((1, 0), **i32), 4, 2)
    assert slots.tolist() == [-1, -1] and counts.tolist() == [0, 0, 2]


# ---------------------------------------------------------------------------
# Paged codec
# ---------------------------------------------------------------------------

def _slots(rng, N, rows, holes):
    s = rng.permutation(rows)[:N].astype(np.int64)
    if holes:
        s[rng.random(N) < 0.3] = -1
        s[N // 2] = rows          # outside the pool: stored nowhere
        s[-1] = -(1 << 40)
    return s


@pytest.mark.parametrize("N,H,holes", [(1, 1, False), (7, 3, True), (33, 8, True), (64, 5, False),
                                       (700, 8, True), (4001, 2, True)])
@pytest.mark.parametrize("d,bits,group,rot", [(64, 4, 16, 0), (64, 8, 64, 1), (128, 4, 16, 0),
                                              (128, 8, 16, 0), (128, 4, 128, 1), (256, 4, 32, 0),
                                              (256, 8, 256, 0), (256, 8, 16, 1)])
def test_paged_codec(N, H, holes, d, bits, group, rot):
    """Codes and scales at the slots match the oracle as the codec's do; every
    other row of the pools keeps its bytes; reading back gives the oracle's
    dequantisation, and rows without a slot keep theirs."""
    import torch
    N = min(N, 10 ** 6 // (H * d))   # the oracle's share of the time
    rng = np.random.default_rng(N * 31 + H * 7 + d + bits + group + rot)
    S, rows = 2, N + 13
    x = rng.standard_normal((S, N, H, d))
    x[..., 3::29] *= 9
    x = x.astype(np.float16)
    signs = np.where(rng.random((S, H, d)) < 0.5, -1, 1).astype(np.int8)
    lam = oracle.calibrate_lambda(x, signs, min(N, 64), rot).astype(np.float32)
    slots = _slots(rng, N, rows, holes)
    live = (slots >= 0) & (slots < rows)
    codes = torch.full((S, rows, H, d * bits // 8), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((S, rows, H, d // group), -3.0, dtype=torch.float16, device=DEV)
    rq.quantize_paged(_t(x), _t(signs), _t(lam), _t(slots), codes, scales, group, bits, rot)
    assert rq.srftq_check_device() == 0
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    rest = np.setdiff1d(np.arange(rows), slots[live])
    assert (c[:, rest] == 0xA5).all() and (s[:, rest] == -3.0).all()
    ref = oracle.quantize(x[:, live], signs, lam, group, bits, rot)
    parity.assert_clean(parity.check_codes(ref, c[:, slots[live]],
                                           s[:, slots[live]].view(np.uint16), bits, group), "codes")

    xhat = torch.full((S, N, H, d), 77.0, dtype=torch.float16, device=DEV)
    got = rq.dequantize_paged(codes, scales, _t(slots), _t(signs), _t(lam), d, group, bits, rot,
                              out=xhat)
    assert rq.srftq_check_device() == 0
    got = got.cpu().numpy()
    assert (got[:, ~live] == 77.0).all()
    want = oracle.dequantize(c[:, slots[live]], s[:, slots[live]].view(np.uint16), signs, lam, d,
                             group, bits, rot)["xhat64"]
    err = np.abs(got[:, live].astype(np.float64) - want) / np.maximum(1.0, np.abs(want))
    assert err.max(initial=0.0) <= parity.DEQ_TOL


def test_paged_codec_windows_and_repeats():
    """x and xhat as windows of a larger buffer; one slot read many times; no
    out given: rows without a slot are zero."""
    import torch
    rng = np.random.default_rng(5)
    S, N, H, d = 2, 50, 4, 128
    big = _t(rng.standard_normal((S, 200, H, d)).astype(np.float16))
    x = big[:, 30:30 + N]
    signs = _t(np.where(rng.random((S, H, d)) < 0.5, -1, 1).astype(np.int8))
    lam = rq.calibrate_lambda(x.contiguous(), signs, N)
    codes = torch.zeros((S, 64, H, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((S, 64, H, d // 16), dtype=torch.float16, device=DEV)
    rq.quantize_paged(x, signs, lam, torch.arange(N, device=DEV), codes, scales)
    want_c, want_s = rq.quantize(x.contiguous(), signs, lam)
    # the same rotation to within rounding: codes may differ next to a border only
    assert (codes[:, :N] != want_c).float().mean() < 1e-3
    torch.testing.assert_close(scales[:, :N], want_s, rtol=2 ** -10, atol=0)
    rep = torch.full((70,), 3, dtype=torch.int64, device=DEV)
    rep[11::7] = -1
    got = rq.dequantize_paged(codes, scales, rep, signs, lam, d)
    one = rq.dequantize(codes[:, 3:4].contiguous(), scales[:, 3:4].contiguous(), signs, lam, d)
    live = rep >= 0
    torch.testing.assert_close(got[:, live], one.expand(S, int(live.sum()), H, d), rtol=2 ** -9,
                               atol=1e-5)
    assert (got[:, ~live] == 0).all()


def test_paged_codec_far_rows():
    """A pool whose byte offsets pass 2^32: the last rows of it."""
    import torch
    rng = np.random.default_rng(6)
    H, d, rows = 8, 128, 9_000_000           # 4.6 GB of codes
    x = _t(rng.standard_normal((1, 40, H, d)).astype(np.float16))
    signs = _t(np.where(rng.random((1, H, d)) < 0.5, -1, 1).astype(np.int8))
    lam = torch.ones((1, H, d), device=DEV)
    codes = torch.empty((1, rows, H, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((1, rows, H, d // 16), dtype=torch.float16, device=DEV)
    slots = rows - 1 - torch.arange(40, device=DEV)
    rq.quantize_paged(x, signs, lam, slots, codes, scales)
    got = rq.dequantize_paged(codes, scales, slots, signs, lam, d)
    c, s = rq.quantize(x, signs, lam)
    want = rq.dequantize(c, s, signs, lam, d)
    err = (got.float() - want.float()).abs()
    assert err.max() < 0.3 and (err > 1e-2).float().mean() < 1e-2   # a code next to a border


# ---------------------------------------------------------------------------
# Shared-prefix attention
# ---------------------------------------------------------------------------

def _attn_case(rng, n_seq, H, g, d, bits, group, rot, prefix, own, page, dtype, q_gain=1.0):
    """Pools, tables and queries; own: own tokens of every sequence, or -k for a
    sequence of only k tokens of the prefix."""
    lens = np.array([prefix + o if o >= 0 else -o - 1 for o in own], np.int64)
    n_prefix = -(-prefix // page)
    shared = prefix // page
    held = np.maximum(-(-lens // page) - shared, 0)
    n_pages = n_prefix + int(held.sum()) + 2
    ids = rng.permutation(n_pages).astype(np.int32)
    width = max(int((-(-lens // page)).max(initial=0)), 1)
    table = np.full((n_seq, width), -1, np.int32)
    at = n_prefix
    for b in range(n_seq):
        k = int(held[b])
        table[b, shared:shared + k] = ids[at:at + k]
        at += k
    kc, ks, ksg, kl, kh = paged.cache(rng, n_pages * page, H, d, bits, group, rot)
    vc, vs, vsg, vl, vh = paged.cache(rng, n_pages * page, H, d, bits, group, rot)
    q = _t((q_gain * rng.standard_normal((n_seq, H * g, d))).astype(np.float32))
    import torch
    q = q.to(getattr(torch, dtype))
    dev = dict(k_codes=_t(kc), k_scales=_t(ks.view(np.float16)), k_signs=_t(ksg), k_lambda=_t(kl),
               v_codes=_t(vc), v_scales=_t(vs.view(np.float16)), v_signs=_t(vsg), v_lambda=_t(vl),
               block_table=_t(table), seq_lens=_t(lens.astype(np.int32)),
               prefix_table=_t(ids[:max(n_prefix, 1)]), prefix_len=prefix, page_size=page,
               group=group, bits=bits, rotation=rot)
    host = dict(khat=kh, vhat=vh, block_table=table, seq_lens=lens, prefix_table=ids[:n_prefix],
                prefix_len=prefix, page=page)
    return q, dev, host


def _check(q, dev, host, lse_tol=8 * paged.U):
    import torch
    out, lse = rq.prefix_attention(q, **dev, return_lse=True)
    assert rq.srftq_check_device() == 0
    ref, ref_lse = paged.attention(q.double().cpu().numpy(), scale=1 / math.sqrt(q.shape[2]),
                                   **host)
    worst = paged.check_attention(out.double().cpu().numpy(), ref, torch.finfo(q.dtype).eps)
    got = lse.double().cpu().numpy()
    assert (np.isneginf(got) == np.isneginf(ref_lse)).all()
    fin = np.isfinite(ref_lse)
    assert np.abs(got[fin] - ref_lse[fin]).max(initial=0.0) <= lse_tol
    return worst


def _ragged(rng, n_seq, most):
    own = rng.integers(0, most + 1, n_seq)
    own[0] = most
    return own


SHAPES = [   # n_seq, H, g, prefix, most own, page
    (1, 1, 1, 0, 1, 16), (1, 2, 1, 1, 0, 16), (3, 2, 2, 37, 5, 16), (2, 1, 8, 0, 129, 1),
    (5, 3, 6, 100, 70, 24), (4, 2, 16, 64, 64, 64), (17, 1, 4, 129, 33, 32), (40, 2, 7, 300, 20, 16),
    (33, 1, 8, 1000, 3, 128), (3, 1, 3, 513, 300, 7), (130, 1, 2, 65, 9, 16),
    # many rows and tokens, for the tcgen05 kernels: one row tile, a full one, three
    (12, 4, 8, 4001, 20, 7), (16, 3, 8, 3203, 5, 1), (40, 2, 7, 3001, 20, 16),
    (33, 1, 8, 6500, 3, 128),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,bits,group,rot,dtype", [
    (128, 4, 16, 0, "float16"), (128, 4, 16, 0, "bfloat16"), (128, 8, 16, 1, "float16"),
    (128, 8, 128, 0, "bfloat16"), (64, 4, 16, 0, "float16"), (64, 8, 32, 1, "bfloat16"),
    (256, 4, 32, 0, "float16"), (256, 8, 64, 0, "bfloat16"), (128, 4, 64, 1, "float16"),
    (256, 4, 256, 1, "bfloat16")])
def test_prefix_attention(shape, d, bits, group, rot, dtype):
    n_seq, H, g, prefix, most, page = shape
    rng = np.random.default_rng(hash(shape) % 1000 + d + bits + group)
    own = _ragged(rng, n_seq, most)
    if n_seq > 2:
        own[1] = -1                                    # no token at all
        own[2] = -1 - prefix // 2                      # half of the prefix
    _check(*_attn_case(rng, n_seq, H, g, d, bits, group, rot, prefix, own, page, dtype))


@pytest.mark.parametrize("n_seq,g", [(2, 1), (48, 8)])
def test_prefix_attention_peaked(n_seq, g):
    """Queries five times as long: scores spread widely and a few tokens carry
    the row, so the running maximum moves often. With two tokens of like weight
    the score errors act on the difference of their values, which the row's own
    size does not bound: each row has its own first-order standard deviation
    (paged.attention). The 10^5 coordinates stay within 6 of it (a normal one
    passes that with probability 2e-9 each; sums of few roundings are narrower)
    plus the output's own rounding, half a step."""
    import torch
    rng = np.random.default_rng(n_seq)
    q, dev, host = _attn_case(rng, n_seq, 2, g, 128, 4, 16, 0, 700 if n_seq == 2 else 3000,
                              _ragged(rng, n_seq, 100), 16,
                              "bfloat16", q_gain=5.0)
    out = rq.prefix_attention(q, **dev).double().cpu().numpy()
    sd = np.zeros((*q.shape[:2], 1))
    ref, _ = paged.attention(q.double().cpu().numpy(), scale=1 / math.sqrt(128), spread=sd, **host)
    tol = torch.finfo(torch.bfloat16).eps / 2 * np.abs(ref) + 6 * sd
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())


def test_prefix_attention_ignores_what_lies_behind():
    """Rows behind the last token, whole unused pages, table entries behind the
    last page and the tables of empty sequences may hold anything: NaN and
    infinite scales, page numbers far outside the pool."""
    import torch
    rng = np.random.default_rng(12)
    n_seq, page = 6, 32
    own = [5, 0, -1, 33, 1, 64]
    for dtype, n_more, prefix in (("float16", 1, 70), ("bfloat16", 40, 70), ("bfloat16", 40, 1254),
                                  ("float16", 20, 1254)):
        case = _attn_case(rng, n_seq * n_more, 2, 4, 128, 4, 16, 0, prefix, own * n_more, page,
                          dtype)
        q, dev, host = case
        used = np.zeros(host["khat"].shape[0], bool)
        t = np.arange(prefix)
        used[paged.rows_of(host["prefix_table"], t, page, 10 ** 6)] = True
        for b in range(len(own) * n_more):
            t = np.arange(prefix, max(int(host["seq_lens"][b]), prefix))
            if t.size:
                used[paged.rows_of(host["block_table"][b], t, page, 10 ** 6)] = True
        bad = _t(~used)
        assert bad.any()
        dev["k_scales"][bad] = float("nan")
        dev["v_scales"][bad] = float("inf")
        table = dev["block_table"].cpu().numpy()
        for b in range(len(table)):
            k = -(-int(host["seq_lens"][b]) // page)
            table[b, k:] = 2 ** 31 - 1
            table[b, :prefix // page] = -(2 ** 31)      # shared entries are not read
        dev["block_table"] = _t(table)
        host["block_table"] = table
        _check(q, dev, host)


def test_prefix_attention_bad_pages():
    """Tokens whose table entry is no page of the pool are left out; sequence
    lengths beyond the table are cut, negative ones are empty."""
    rng = np.random.default_rng(13)
    q, dev, host = _attn_case(rng, 5, 1, 2, 128, 4, 16, 0, 64, [40, 10, 50, 3, 20], 16, "float16")
    table = dev["block_table"].cpu().numpy()
    table[0, 5] = -1
    table[2, 4] = 10 ** 9
    table[2, 6] = -(2 ** 31)
    pt = dev["prefix_table"].cpu().numpy()
    pt[1] = -4
    lens = dev["seq_lens"].cpu().numpy()
    lens[3] = 2 ** 31 - 1
    lens[4] = -9
    for k, v in (("block_table", table), ("prefix_table", pt), ("seq_lens", lens)):
        dev[k] = _t(v)
        host[k] = v
    _check(q, dev, host)


@pytest.mark.parametrize("d,bits,dtype,g", [
    (128, 4, "float16", 2), (64, 8, "bfloat16", 1),      # few query rows
    (128, 4, "float16", 8), (128, 8, "float16", 8), (64, 4, "bfloat16", 8),   # up to 128 rows
    (128, 4, "bfloat16", 16), (64, 8, "bfloat16", 12),   # two row tiles
    (256, 4, "float16", 16), (256, 8, "bfloat16", 12), (256, 4, "bfloat16", 1)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_prefix_attention_non_finite_prefix_token(d, bits, dtype, g, what):
    """Scales of prefix tokens that are NaN or infinite reach the sequences that
    attend to them and no other, though all share the tiles they lie in: of those
    that end before, every bit is as without."""
    rng = np.random.default_rng(d + bits + g)
    n_seq, prefix = 14, 4800
    own = [3, -1 - 200, -1 - 203, 0, -1 - 64, -1 - 5, 60, -1 - 201, -1, -1 - 4799, -1 - 4799, 1, 2,
           -1 - 202]
    q, dev, host = _attn_case(rng, n_seq, 2, g, d, bits, 16, 0, prefix, own, 16, dtype)
    want = rq.prefix_attention(q, **dev)
    row = lambda t: int(paged.rows_of(host["prefix_table"], np.array([t]), 16, 10 ** 6)[0])
    scales = dev[what + "_scales"]
    scales[row(201), 1, 3] = float("nan")        # head 1 only
    scales[row(250), 1, 0] = float("inf")
    scales[row(4799), 1] = float("-inf")
    got = rq.prefix_attention(q, **dev)
    assert rq.srftq_check_device() == 0
    hit = _t(np.asarray(host["seq_lens"]) > 201)
    assert bool((got[:, :g] == want[:, :g]).all())          # head 0
    assert bool((got[~hit] == want[~hit]).all())
    assert not bool(got[hit][:, g:].isfinite().any())


@pytest.mark.parametrize("n_seq,prefix,bits,d,dtype", [
    (3, 100, 4, 128, "float16"), (3, 100, 8, 64, "float16"), (20, 6600, 4, 128, "float16"),
    (50, 6600, 4, 64, "bfloat16"), (30, 6600, 4, 256, "float16"), (20, 6600, 8, 128, "float16")])
def test_prefix_attention_small_scales(n_seq, prefix, bits, d, dtype):
    """Scales 2^-9 (int8: 2^-5) of the usual ones, with lambda as much larger:
    the same vectors, so the same result. The values keep their bits as long as
    their scale is a normal number."""
    rng = np.random.default_rng(n_seq + bits + d)
    q, dev, host = _attn_case(rng, n_seq, 2, 4, d, bits, 16, 0, prefix, _ragged(rng, n_seq, 90), 16,
                              dtype)
    k = 9 if bits == 4 else 5
    for c in "kv":
        small = dev[c + "_scales"].float() * 2.0 ** -k
        assert bool((small.half().float() == small).all())
        dev[c + "_scales"] = small.half()
        dev[c + "_lambda"] = dev[c + "_lambda"] * 2.0 ** k
    _check(q, dev, host)


def test_prefix_attention_all_pages_bad():
    """No token of a sequence has a page: zeros and -inf, as without tokens."""
    rng = np.random.default_rng(14)
    q, dev, host = _attn_case(rng, 3, 2, 3, 64, 8, 16, 0, 20, [9, 4, 0], 16, "bfloat16")
    dev["block_table"].fill_(-1)
    dev["prefix_table"].fill_(-1)
    out, lse = rq.prefix_attention(q, **dev, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("prefix", [200, 7000])
def test_prefix_attention_non_finite_query(prefix):
    """A NaN in one query stays in that query's output."""
    import torch
    rng = np.random.default_rng(15)
    q, dev, host = _attn_case(rng, 40, 1, 4, 128, 4, 16, 0, prefix, _ragged(rng, 40, 30), 16,
                              "float16")
    want = rq.prefix_attention(q, **dev)
    q2 = q.clone()
    q2[7, 2, 5] = float("nan")
    got = rq.prefix_attention(q2, **dev)
    assert got[7, 2].isnan().all()
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[7, 2] = False
    assert torch.equal(got[keep.to(DEV)], want[keep.to(DEV)])


def test_prefix_split_does_not_matter():
    """The same tokens as a prefix, or as every sequence's own pages."""
    rng = np.random.default_rng(16)
    q, dev, host = _attn_case(rng, 9, 2, 4, 128, 4, 16, 0, 256, _ragged(rng, 9, 90), 32, "bfloat16")
    table = dev["block_table"].cpu().numpy()
    table[:, :8] = dev["prefix_table"].cpu().numpy()[:8]
    host["block_table"] = table
    dev["block_table"] = _t(table)
    for prefix in (256, 0, 64, 100):
        dev["prefix_len"] = host["prefix_len"] = prefix
        _check(q, dev, host)


def test_prefix_attention_far_rows():
    """Pages whose byte offsets pass 2^32: the pool's last pages against a copy
    of the same rows in a small pool."""
    import torch
    rng = np.random.default_rng(17)
    page, rows, small = 64, 9_000_000 // 64 * 64, 640
    q, dev, _ = _attn_case(rng, 3, 8, 2, 128, 4, 16, 0, 300, [100, 90, 80], page, "float16")
    want = rq.prefix_attention(q, **dev)
    n = dev["k_codes"].shape[0]
    big = {}
    for k in ("k_codes", "k_scales", "v_codes", "v_scales"):
        big[k] = torch.empty((rows, *dev[k].shape[1:]), dtype=dev[k].dtype, device=DEV)
        big[k][rows - n:] = dev[k]
    off = (rows - n) // page
    big["block_table"] = dev["block_table"] + off
    big["prefix_table"] = dev["prefix_table"] + off
    got = rq.prefix_attention(q, **{**dev, **big})
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# Streams, graphs and the run of all three
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("prefix", [130, 50_003])
def test_other_stream_and_graphs(prefix):
    """A call on another stream, and two captured graphs with a workspace each,
    replayed with new lengths and queries in the same buffers."""
    import torch
    rng = np.random.default_rng(18)
    q, dev, host = _attn_case(rng, 6, 2, 4, 128, 4, 16, 0, prefix, [60, 9, 0, 33, 1, 64], 16,
                              "float16")
    want = rq.prefix_attention(q, **dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rq.prefix_attention(q, **dev, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    desc = rq.make_desc(128, 2, 16, 4)
    ws = [torch.empty(rq.srftq_prefix_attention_workspace(desc, 6, 4, prefix), dtype=torch.uint8,
                      device=DEV) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    for w, o in zip(ws, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            rq.prefix_attention(q, **dev, workspace=w, out=o)
        graphs.append(gr)
    q.copy_(q.flip(0))
    dev["seq_lens"].copy_(dev["seq_lens"].flip(0))
    dev["block_table"].copy_(dev["block_table"].flip(0))
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want.flip(0))


@pytest.mark.parametrize("dtype,n_seq,d,prefix", [
    ("bfloat16", 40, 128, 6600), ("float16", 20, 64, 6600), ("float16", 3, 128, 300),
    ("bfloat16", 24, 256, 6600), ("bfloat16", 40, 64, 300)])
def test_one_workspace_for_calls_in_turn(dtype, n_seq, d, prefix):
    """Calls in a stream may share a workspace: two batches in turn, thirty
    times without a wait between, with the results they have by themselves."""
    import torch
    rng = np.random.default_rng(20)
    cases = [_attn_case(rng, n_seq, 2, 4, d, 4, 16, 0, prefix,
                        _ragged(rng, n_seq, 200 - 150 * i), 16, dtype)[:2] for i in range(2)]
    want = [rq.prefix_attention(q, **dev) for q, dev in cases]
    need = rq.srftq_prefix_attention_workspace(rq.make_desc(d, 2, 16, 4), n_seq, 4, prefix)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device=DEV)   # whatever it holds
    got = [rq.prefix_attention(q, **dev, workspace=ws) for _ in range(30) for q, dev in cases]
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    assert rq.srftq_check_device() == 0


@pytest.mark.parametrize("prefix,n_seq", [(64, 6), (6400, 20)])
def test_tokens_written_between_calls(prefix, n_seq):
    """Tokens are written into pages between calls, in place beside ones that the
    call before has read: as with copies of pools and tables at other addresses."""
    import torch
    rng = np.random.default_rng(23)
    H, d, page = 2, 128, 16
    q, dev, _ = _attn_case(rng, n_seq, H, 4, d, 4, 16, 0, prefix, [40] * n_seq, page, "bfloat16")
    i32 = dict(dtype=torch.int32, device=DEV)
    dev["seq_lens"] = torch.full((n_seq,), prefix + 20, **i32)
    table = dev["block_table"].long()
    b = torch.arange(n_seq, device=DEV)
    for t in range(prefix + 20, prefix + 40):
        slots = table[b, t // page] * page + t % page
        for c in "kv":
            x = torch.randn((1, n_seq, H, d), device=DEV).half()
            rq.quantize_paged(x, dev[c + "_signs"][None], dev[c + "_lambda"][None], slots,
                              dev[c + "_codes"][None], dev[c + "_scales"][None])
        dev["seq_lens"] += 1
        got = rq.prefix_attention(q, **dev)
        fresh = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in dev.items()}
        assert torch.equal(got, rq.prefix_attention(q, **fresh)), t
    assert rq.srftq_check_device() == 0


def test_two_streams_at_once():
    """Calls on two streams at the same time, each with the workspace that the
    call allocates for itself."""
    import torch
    rng = np.random.default_rng(21)
    cases = [_attn_case(rng, 30, 2, 4, 128, 4, 16, 0, 4000, _ragged(rng, 30, 90), 16, "bfloat16")[:2]
             for _ in range(2)]
    want = [rq.prefix_attention(q, **dev) for q, dev in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, (q, dev) in enumerate(cases):
            got[i].append(rq.prefix_attention(q, **dev, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])


def test_captured_step():
    """Tables, codes and attention of a step captured together and replayed with
    other lengths and vectors in the same buffers, a padded batch among them."""
    import torch
    rng = np.random.default_rng(22)
    H, g, d, page, n_seq, pages = 2, 4, 128, 16, 6, 200
    i32 = dict(dtype=torch.int32, device=DEV)
    signs = _t(np.where(rng.random((2, H, d)) < 0.5, -1, 1).astype(np.int8))
    lam = torch.rand((2, H, d), device=DEV) + 0.5
    table0 = torch.arange(n_seq * 12, **i32).view(n_seq, 12)

    def buffers():
        return dict(codes=torch.zeros((2, pages * page, H, d // 2), dtype=torch.uint8, device=DEV),
                    scales=torch.zeros((2, pages * page, H, d // 16), dtype=torch.float16, device=DEV),
                    table=torch.cat([table0, torch.full((n_seq, 8), -1, **i32)], 1).contiguous(),
                    cached=torch.zeros(n_seq, **i32), new=torch.zeros(n_seq, **i32),
                    free=torch.zeros(40, **i32),
                    x=torch.zeros((2, 160, H, d), dtype=torch.float16, device=DEV),
                    q=torch.zeros((n_seq, H * g, d), dtype=torch.bfloat16, device=DEV))

    def step(b):
        slots, lens, _, _ = rq.block_tables(b["cached"], b["new"], b["free"], b["table"], page, 160)
        rq.quantize_paged(b["x"], signs, lam, slots, b["codes"], b["scales"])
        return rq.prefix_attention(b["q"], b["codes"][0], b["scales"][0], signs[0], lam[0],
                                   b["codes"][1], b["scales"][1], signs[1], lam[1], b["table"], lens,
                                   page_size=page)

    graphed, eager = buffers(), buffers()
    step(graphed)                                # what the first call of a kernel sets up
    for k, v in buffers().items():
        graphed[k].copy_(v)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step(graphed)
    cached = np.array([192, 100, 7, 0, 191, 33])
    for it in range(3):
        new = np.array([[9, 0, 40, 16, 1, 3], [1, 1, 1, 0, 1, 1], [0, 20, 0, 0, 5, 0]][it])
        feed = dict(cached=_t(cached.astype(np.int32)), new=_t(new.astype(np.int32)),
                    free=torch.arange(n_seq * 12 + 40 * it, n_seq * 12 + 40 * it + 40, **i32),
                    x=_t(rng.standard_normal((2, 160, H, d)).astype(np.float16)),
                    q=_t(rng.standard_normal((n_seq, H * g, d)).astype(np.float32)).bfloat16())
        for b in (graphed, eager):
            for k, v in feed.items():
                b[k].copy_(v)
        gr.replay()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(graphed["table"], eager["table"])
        assert torch.equal(graphed["codes"], eager["codes"])
        cached = cached + new
    assert rq.srftq_check_device() == 0


def test_serving_loop():
    """As a server uses them: prompts in, then tokens one by one, over a shared
    document; tables, slots, codes and attention all from the device's own
    outputs, against attention over the dequantised vectors that went in."""
    import torch
    rng = np.random.default_rng(19)
    H, g, d, page, group, bits = 2, 4, 128, 16, 16, 4
    n_seq, doc = 5, 83
    n_pages = 64
    pool_c = torch.zeros((2, n_pages * page, H, d * bits // 8), dtype=torch.uint8, device=DEV)
    pool_s = torch.zeros((2, n_pages * page, H, d // group), dtype=torch.float16, device=DEV)
    signs = _t(np.where(rng.random((2, H, d)) < 0.5, -1, 1).astype(np.int8))
    free = _t(rng.permutation(n_pages).astype(np.int32))
    i32 = dict(dtype=torch.int32, device=DEV)

    def kv(n):
        return _t(rng.standard_normal((2, n, H, d)).astype(np.float16))

    lam = rq.calibrate_lambda(kv(512), signs)
    # the document: one sequence, its own table
    doc_table = torch.full((1, 8), -1, **i32)
    slots, _, _, counts = rq.block_tables(torch.zeros(1, **i32), torch.tensor([doc], **i32), free,
                                          doc_table, page, doc)
    x_doc = kv(doc)
    rq.quantize_paged(x_doc, signs, lam, slots, pool_c, pool_s)
    used = int(counts[0])
    seen = [[x_doc] for _ in range(n_seq)]
    # every sequence starts with the document's full pages and a copy of its last part
    full = doc // page
    table = torch.full((n_seq, 24), -1, **i32)
    table[:, :full] = doc_table[0, :full]
    lens = torch.full((n_seq,), full * page, **i32)
    tail = x_doc[:, full * page:]
    first = True
    for step in range(4):
        new = (torch.full((n_seq,), doc - full * page, **i32) if first else
               torch.tensor([7, 0, 1, 20, 3] if step == 1 else [1, 1, 0, 1, 1], **i32))
        n = int(new.sum())
        batch = n + 3                                   # a padded batch
        slots, lens, starts, counts = rq.block_tables(lens, new, free[used:], table, page, batch)
        used += int(counts[0])
        if first:
            x = torch.cat([tail] * n_seq + [kv(3)], 1)
        else:
            x = kv(batch)
            for b in range(n_seq):
                seen[b].append(x[:, int(starts[b]):int(starts[b + 1])])
        rq.quantize_paged(x, signs, lam, slots, pool_c, pool_s)
        first = False
        q = _t(rng.standard_normal((n_seq, H * g, d)).astype(np.float16))
        out = rq.prefix_attention(q, pool_c[0], pool_s[0], signs[0], lam[0], pool_c[1], pool_s[1],
                                  signs[1], lam[1], table, lens, doc_table[0], doc, page_size=page)
        assert rq.srftq_check_device() == 0
        for b in range(n_seq):
            xs = torch.cat(seen[b], 1).contiguous()
            assert xs.shape[1] == int(lens[b])
            c, s = rq.quantize(xs, signs, lam)
            hat = oracle.dequantize(c.cpu().numpy(), s.cpu().numpy().view(np.uint16),
                                    signs.cpu().numpy(), lam.cpu().numpy(), d, group, bits,
                                    0)["xhat64"]
            for hq in range(H * g):
                sc = hat[0, :, hq // g] @ q[b, hq].double().cpu().numpy() / math.sqrt(d)
                p = np.exp(sc - sc.max())
                ref = p @ hat[1, :, hq // g] / p.sum()
                got = out[b, hq].double().cpu().numpy()
                # a code next to a border may fall either way: one step of one of
                # xs.shape[1] * d codes, far below this part of the row's norm
                assert np.linalg.norm(got - ref) <= 0.01 * np.linalg.norm(ref)


@pytest.mark.parametrize("d,bits,group,dtype", [(128, 8, 16, "bfloat16"), (128, 4, 16, "float16"),
                                                (64, 4, 16, "bfloat16"), (256, 4, 32, "bfloat16"),
                                                (256, 8, 32, "float16")])
def test_prefix_attention_long(d, bits, group, dtype):
    """A prefix of many tiles per part, on every kind of tile, ten times over:
    the same bits every time, no guard, and the reference's values (in torch, 64
    bits, from this library's own dequantisation before its fp16 rounding is
    replaced by the scales and codes)."""
    import torch
    gen = torch.Generator(device=DEV).manual_seed(d + bits)
    n_seq, H, g, prefix, page = 9, 16, 8, 40_000, 64
    rows = -(-prefix // page) * page
    pools = {}
    for kv in "kv":
        c = torch.randint(0, 256, (rows, H, d * bits // 8), generator=gen, device=DEV,
                          dtype=torch.int32).to(torch.uint8)
        s = torch.rand((rows, H, d // group), generator=gen, device=DEV) * 0.29 + 0.01
        pools[kv] = (c, (s / (16 if bits == 8 else 1)).to(torch.float16))
    ones = torch.ones((H, d), dtype=torch.int8, device=DEV)
    lam = torch.ones((H, d), device=DEV)
    q = torch.randn((n_seq, H * g, d), generator=gen, device=DEV).to(getattr(torch, dtype))
    lens = torch.full((n_seq,), prefix, dtype=torch.int32, device=DEV)
    lens[3] = 17_001
    table = torch.zeros((n_seq, 1), dtype=torch.int32, device=DEV)
    pt = torch.randperm(rows // page, generator=gen, device=DEV).to(torch.int32)
    call = lambda: rq.prefix_attention(  # noqa: E731
        q, *pools["k"], ones, lam, *pools["v"], ones, lam, table, lens, pt, prefix, page_size=page,
        group=group, bits=bits, rotation=rq.SRHT)
    out = call()
    assert rq.srftq_check_device() == 0
    for _ in range(10):
        assert torch.equal(call(), out)
    assert rq.srftq_check_device() == 0
    # SRHT without signs is its own inverse, orthogonal: scores and values in the
    # rotated domain, rotated back by the Hadamard matrix
    i = torch.arange(d, device=DEV)
    had = i[:, None] & i[None, :]
    had = 1 - 2 * sum((had >> b) & 1 for b in range(8)).remainder(2).double()
    had /= math.sqrt(d)
    t = torch.arange(prefix, device=DEV)
    at = pt[t // page].long() * page + t % page

    def values(c, s, h):
        c = c[at, h].long()
        if bits == 8:
            c = torch.where(c > 127, c - 256, c)
        else:
            c = torch.stack((c % 16, c // 16), -1).flatten(-2)
            c = torch.where(c > 7, c - 16, c)
        return c.double() * s[at, h].double().repeat_interleave(group, -1)

    for h in (0, 7, H - 1):
        k, v = values(*pools["k"], h), values(*pools["v"], h)
        qh = q[:, h * g:(h + 1) * g].double() @ had
        sc = qh @ k.T / math.sqrt(d)
        sc.masked_fill_((t >= lens[:, None])[:, None], -math.inf)
        ref = torch.softmax(sc, -1) @ v @ had
        paged.check_attention(out[:, h * g:(h + 1) * g].double().cpu().numpy(), ref.cpu().numpy(),
                              torch.finfo(q.dtype).eps)
