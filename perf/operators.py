"""The paged-cache operators of this library as measured cases.

Three operators that a serving loop runs next to one another on a cache of
quantised keys and values:

- ``tables``     block tables and slot maps of a step, from request lengths;
- ``codec``      new vectors quantised into the pages' slots, and slots read back;
- ``attention``  one decode step over the pages, for a batch that shares a prefix.

A cache is a pool of rows, ``page`` consecutive rows to a page; a row holds
``heads`` vectors of ``d`` coordinates as codes of 4 or 8 bits and one fp16
scale for each ``group`` coordinates of the rotated, rescaled vector.
"""

import math

import numpy as np
import torch

own = False

F32, F64 = torch.float32, torch.float64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the step of a small decode batch: one token for each request
        {"name": "tables_decode", "op": "tables", "n_seq": 32, "cached": 32768, "new": 1, "page": 64},
        # a batch of prompts of all lengths, short pages, some requests with nothing new
        {"name": "tables_prompts", "op": "tables", "n_seq": 2047, "cached": 300, "new": 900, "page": 16},
        # one decoded token of 32 sequences, K and V of one layer
        {"name": "append_tokens", "op": "codec", "rows": 32, "heads": 8, "d": 128, "bits": 4,
         "group": 16, "rotation": "srft", "page": 64, "padded": 0},
        # a prompt of wide heads
        {"name": "prompt_wide", "op": "codec", "rows": 8192, "heads": 4, "d": 256, "bits": 4,
         "group": 32, "rotation": "srft", "page": 32, "padded": 0},
        # a long prompt in 8 bits, the last rows of the batch being padding
        {"name": "prompt_int8", "op": "codec", "rows": 65536, "heads": 8, "d": 128, "bits": 8,
         "group": 16, "rotation": "srft", "page": 64, "padded": 100},
        # a few chats behind one short system prompt, two KV heads
        {"name": "chat_few", "op": "attention", "n_seq": 4, "heads": 2, "q_per_kv": 6, "d": 128,
         "bits": 4, "group": 16, "rotation": "srft", "prefix": 509, "suffix": 64, "page": 16,
         "dtype": "float16"},
        # the ordinary serving batch behind a shared document
        {"name": "chat_batch", "op": "attention", "n_seq": 32, "heads": 8, "q_per_kv": 4, "d": 128,
         "bits": 4, "group": 16, "rotation": "srft", "prefix": 8192, "suffix": 1024, "page": 64,
         "dtype": "bfloat16"},
        # a decode stream of 32768 tokens whose batch shares most of its context
        {"name": "long_stream", "op": "attention", "n_seq": 32, "heads": 8, "q_per_kv": 1, "d": 128,
         "bits": 4, "group": 16, "rotation": "srft", "prefix": 28672, "suffix": 4096, "page": 64,
         "dtype": "float16"},
        # wide heads, few sequences
        {"name": "wide_heads", "op": "attention", "n_seq": 4, "heads": 4, "q_per_kv": 2, "d": 256,
         "bits": 4, "group": 32, "rotation": "srft", "prefix": 8192, "suffix": 777, "page": 32,
         "dtype": "float16"},
        # a long context in 8 bits
        {"name": "long_int8", "op": "attention", "n_seq": 16, "heads": 8, "q_per_kv": 8, "d": 128,
         "bits": 8, "group": 16, "rotation": "srht", "prefix": 131072, "suffix": 333, "page": 128,
         "dtype": "bfloat16"},
        # nothing shared: plain paged decoding of ragged sequences
        {"name": "paged_only", "op": "attention", "n_seq": 64, "heads": 8, "q_per_kv": 2, "d": 64,
         "bits": 4, "group": 16, "rotation": "srft", "prefix": 0, "suffix": 2048, "page": 16,
         "dtype": "float16"},
        # the largest batch: many samples of one long prompt
        {"name": "many_samples", "op": "attention", "n_seq": 128, "heads": 8, "q_per_kv": 8, "d": 128,
         "bits": 4, "group": 16, "rotation": "srft", "prefix": 32768, "suffix": 1500, "page": 64,
         "dtype": "bfloat16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "codec", "attention", "attention"])
    while True:   # sizes again until the case costs no more than the largest listed one
        if op == "tables":
            case = {"op": op, "n_seq": _log(rng, 1, 4096), "cached": _log(rng, 1, 40000),
                    "new": _log(rng, 1, 4000), "page": rng.choice([1, 16, 24, 32, 64, 128, 256])}
        else:
            d = rng.choice([64, 128, 128, 256])
            case = {"op": op, "heads": rng.choice([1, 2, 3, 4, 5, 8]), "d": d,
                    "bits": rng.choice([4, 4, 8]),
                    "group": rng.choice([g for g in (16, 16, 32, 64, 128) if g <= d]),
                    "rotation": rng.choice(["srft", "srft", "srht"]),
                    "page": rng.choice([16, 24, 32, 64, 128, 256])}
            if op == "codec":
                rows = _log(rng, 1, 65536)
                case.update(rows=rows, padded=rng.choice([0, rows // 7]))
            else:
                case.update(n_seq=_log(rng, 1, 128), q_per_kv=rng.choice([1, 2, 3, 4, 6, 7, 8, 16]),
                            prefix=rng.choice([0, _log(rng, 1, 131072), _log(rng, 16, 32768)]),
                            suffix=_log(rng, 1, 4096), dtype=rng.choice(["float16", "bfloat16"]))
        w, size = work(case), _touched(case)
        top = [c for c in listed() if c["op"] == op]
        if (w["bytes"] <= max(work(c)["bytes"] for c in top)
                and w["flops"] <= max(work(c)["flops"] for c in top)
                and size <= max(_touched(c) for c in top)):
            return case


def _new_lens(case):
    """Cached and new tokens of every request: a fixed ragged pattern of the case alone."""
    b = np.arange(case["n_seq"], dtype=np.float64)
    cached = np.floor((b * 0.6180339887498949) % 1.0 * (case["cached"] + 1)).astype(np.int64)
    new = 1 + np.floor((b * 0.7548776662466927) % 1.0 * case["new"]).astype(np.int64)
    if case["new"] > 1:  # decode batches have a token each; mixed ones some idle requests
        new[5::9] = 0
    return cached, new


def _seq_lens(case):
    """Tokens of every sequence, the prefix included: ragged, some with the prefix
    alone, and padding rows without any token."""
    b = np.arange(case["n_seq"], dtype=np.float64)
    own_part = np.ceil((0.37 + b * 0.6180339887498949) % 1.0 * case["suffix"]).astype(np.int64)
    own_part[3::11] = 0
    lens = case["prefix"] + own_part
    lens[13::16] = 0
    return lens


def _pages_up(n, page):
    return -(-n // page)


def _touched(case):
    """Values that the plain form holds at its largest, for draw()'s bound."""
    if case["op"] == "tables":
        cached, new = _new_lens(case)
        return int(new.sum()) + case["n_seq"] * int(_pages_up(cached + new, case["page"]).max())
    if case["op"] == "codec":
        return 2 * case["rows"] * case["heads"] * case["d"]
    rows = case["n_seq"] * case["heads"] * case["q_per_kv"]
    kv = (case["prefix"] + case["n_seq"] * case["suffix"]) * case["heads"] * case["d"]
    return rows * (case["prefix"] + case["suffix"]) + kv


def work(case):
    if case["op"] == "tables":
        cached, new = _new_lens(case)
        taken = _pages_up(cached + new, case["page"]) - _pages_up(cached, case["page"])
        n = case["n_seq"]
        # lengths in; free pages in, table entries out; slots, lengths and row starts out
        return {"bytes": int(8 * n + 8 * taken.sum() + 8 * new.sum() + 8 * n + 16), "flops": 0}
    vec = case["d"] * case["bits"] // 8 + 2 * (case["d"] // case["group"])
    if case["op"] == "codec":
        n = 2 * (case["rows"] - case["padded"]) * case["heads"]
        fft = 2.5 * case["d"] * math.log2(case["d"])
        # vectors in, codes and scales out; codes and scales in, vectors out; slots twice
        return {"bytes": n * (4 * case["d"] + 2 * vec) + 16 * case["rows"], "flops": 2 * n * fft}
    lens = _seq_lens(case)
    own_part = int(np.maximum(lens - case["prefix"], 0).sum())
    shared = case["prefix"] if (lens > 0).any() else 0
    q = case["n_seq"] * case["heads"] * case["q_per_kv"] * case["d"]
    return {"bytes": 2 * vec * case["heads"] * (shared + own_part) + 4 * q,
            "flops": 4 * case["d"] * case["heads"] * case["q_per_kv"] * int(lens.sum())}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rotation_matrix(kind, d, device):
    """R in 64 bits: row j gives packed coordinate j of the rotated vector (before the signs)."""
    i = torch.arange(d, device=device)
    if kind == "srht":
        both = i[:, None] & i[None, :]
        for_bits = (both[..., None] >> torch.arange(8, device=device)) & 1
        return (1 - 2 * (for_bits.sum(-1) & 1)).to(F64) / math.sqrt(d)
    k = i // 2
    angle = (k[:, None] * i[None, :] % d).to(F64) * (2 * math.pi / d)
    rows = torch.where((i % 2 == 0)[:, None], torch.cos(angle), -torch.sin(angle)) * math.sqrt(2 / d)
    rows[0] = 1 / math.sqrt(d)
    rows[1] = (1 - 2 * (i % 2)).to(F64) / math.sqrt(d)
    return rows


def _quantize(x, R, signs, lam, group, bits):
    """x [S, N, H, d] -> codes (whole numbers) and fp16 scales."""
    S, N, H, d = x.shape
    qmax = 2 ** (bits - 1) - 1
    w = (x.to(F32) * signs[:, None].to(F32)) @ R.to(F32).T / lam[:, None]
    g = w.view(S, N, H, d // group, group)
    sigma = (g.abs().amax(-1) / qmax).clamp(max=65504.0).to(torch.float16)
    s = sigma.to(F32)[..., None]
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, 1)), 0).clamp(-qmax, qmax)
    return q.view(S, N, H, d).to(torch.int8), sigma


def _pack(q, bits):
    """Codes as the cache holds them: int8 bytes, or two 4-bit codes to a byte."""
    u = q.view(torch.uint8)
    return u if bits == 8 else (u[..., 0::2] & 15) | (u[..., 1::2] << 4)


def _unpack(codes, bits):
    c = codes.view(torch.int8)
    if bits == 8:
        return c
    return torch.stack(((c << 4) >> 4, c >> 4), -1).flatten(-2)


def _dequantize(codes, scales, R, signs, lam, group, bits):
    """[..., H, bytes] codes and [..., H, groups] scales -> [..., H, d] in 32 bits."""
    y = _unpack(codes, bits).to(F32) * scales.to(F32).repeat_interleave(group, -1) * lam
    return (y @ R.to(F32)) * signs.to(F32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s = {"case": case}
    page = case["page"]
    if case["op"] == "tables":
        cached, new = _new_lens(case)
        held, total = _pages_up(cached, page), _pages_up(cached + new, page)
        n_pages = int(total.sum()) + 7
        ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        width = int(total.max()) + 1
        col = torch.arange(width, device=dev)
        h = torch.from_numpy(held).to(dev)
        start = h.cumsum(0) - h
        at = (start[:, None] + col).clamp(max=n_pages - 1)
        s["block_table"] = torch.where(col < h[:, None], ids[at], -1).to(torch.int32).contiguous()
        s["free_pages"] = ids[int(held.sum()):].contiguous()
        s["cached"] = torch.from_numpy(cached).to(dev, torch.int32)
        s["new"] = torch.from_numpy(new).to(dev, torch.int32)
        s["n_slots"] = int(new.sum()) + 5   # a batch padded by a few rows
        return s

    H, d, group, bits = case["heads"], case["d"], case["group"], case["bits"]
    R = _rotation_matrix(case["rotation"], d, dev)
    s["R"] = R
    s["signs"] = (1 - 2 * torch.randint(0, 2, (2, H, d), generator=gen, device=dev)).to(torch.int8)
    # each channel with a spread of its own, a few of them large, as keys have
    spread = torch.exp(0.3 * normal(2, 1, H, d))
    spread[..., 5::61] *= 8

    def vectors(n):
        return (normal(2, n, H, d) * spread).to(torch.float16)

    sample = vectors(512)
    y = (sample.to(F32) * s["signs"][:, None].to(F32)) @ R.to(F32).T
    s["lam"] = y.square().mean(1).sqrt().contiguous()
    if case["op"] == "codec":
        n = case["rows"]
        rows = _pages_up(n, page) * page
        s["x"] = vectors(n)
        pages = torch.randperm(rows // page, generator=gen, device=dev)
        t = torch.arange(n, device=dev)
        slots = pages[t // page] * page + t % page
        slots[n - case["padded"]:] = -1
        s["slots"] = slots
        s["codes"] = torch.zeros((2, rows, H, d * bits // 8), dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros((2, rows, H, d // group), dtype=torch.float16, device=dev)
        s["xhat"] = torch.zeros((2, n, H, d), dtype=torch.float16, device=dev)
        return s

    lens = _seq_lens(case)
    shared = case["prefix"] // page   # whole pages are shared; a last part has a copy for each
    width = int(_pages_up(np.maximum(lens, case["prefix"]), page).max()) + 1
    mine = np.maximum(_pages_up(lens, page) - shared, 0)
    n_pages = _pages_up(case["prefix"], page) + int(mine.sum()) + 1
    rows = n_pages * page
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    n_prefix = _pages_up(case["prefix"], page)
    s["prefix_table"] = ids[:max(n_prefix, 1)].contiguous()
    m = torch.from_numpy(mine).to(dev)
    col = torch.arange(width, device=dev)
    at = (n_prefix + (m.cumsum(0) - m)[:, None] + col - shared).clamp(0, n_pages - 1)
    table = torch.where(col < shared, ids[col.clamp(max=n_pages - 1)], ids[at])
    held = torch.from_numpy(_pages_up(lens, page)).to(dev)
    s["block_table"] = torch.where(col < held[:, None], table, -1).to(torch.int32).contiguous()
    s["seq_lens"] = torch.from_numpy(lens).to(dev, torch.int32)
    parts = [_quantize(vectors(min(32768, rows - r)), R, s["signs"], s["lam"], group, bits)
             for r in range(0, rows, 32768)]
    codes = torch.cat([_pack(q, bits) for q, _ in parts], 1)
    scales = torch.cat([sc for _, sc in parts], 1)
    s["k_codes"], s["v_codes"] = codes[0].contiguous(), codes[1].contiguous()
    s["k_scales"], s["v_scales"] = scales[0].contiguous(), scales[1].contiguous()
    del parts, codes, scales
    s["sign_k"], s["sign_v"] = s["signs"][0].contiguous(), s["signs"][1].contiguous()
    s["lam_k"], s["lam_v"] = s["lam"][0].contiguous(), s["lam"][1].contiguous()
    # queries with the spread that gives scores of order one
    q = normal(case["n_seq"], H, case["q_per_kv"], d) / spread[0, 0][:, None]
    s["q"] = q.reshape(case["n_seq"], -1, d).to(getattr(torch, case["dtype"]))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"tables": _plain_tables, "codec": _plain_codec, "attention": _plain_attention}[case["op"]](s, case)


def _own(s, case):
    import rotate_then_quantize_b200 as rq

    if case["op"] == "tables":
        slots, seq_lens, row_start, counts = rq.block_tables(
            s["cached"], s["new"], s["free_pages"], s["block_table"], case["page"], s["n_slots"])
        return {"block_table": s["block_table"], "slots": slots, "seq_lens": seq_lens,
                "row_start": row_start, "counts": counts}
    rot = rq.SRFT if case["rotation"] == "srft" else rq.SRHT
    if case["op"] == "codec":
        rq.quantize_paged(s["x"], s["signs"], s["lam"], s["slots"], s["codes"], s["scales"],
                          group=case["group"], bits=case["bits"], rotation=rot)
        return rq.dequantize_paged(s["codes"], s["scales"], s["slots"], s["signs"], s["lam"],
                                   case["d"], group=case["group"], bits=case["bits"], rotation=rot,
                                   out=s["xhat"])
    return rq.prefix_attention(s["q"], s["k_codes"], s["k_scales"], s["sign_k"], s["lam_k"],
                               s["v_codes"], s["v_scales"], s["sign_v"], s["lam_v"],
                               s["block_table"], s["seq_lens"], s["prefix_table"], case["prefix"],
                               page_size=case["page"], group=case["group"], bits=case["bits"],
                               rotation=rot)


def _plain_tables(s, case):
    page, table, free = case["page"], s["block_table"], s["free_pages"]
    cached, new = s["cached"].long(), s["new"].long()
    total = cached + new
    first, last = (cached + page - 1) // page, (total + page - 1) // page
    taken = last - first
    start = taken.cumsum(0) - taken
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= first[:, None]) & (col < last[:, None])
    index = (start[:, None] + col - first[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[index], table)
    row_start = torch.cat((new.new_zeros(1), new.cumsum(0)))
    r = torch.arange(s["n_slots"], device=table.device)
    b = torch.searchsorted(row_start, r, right=True) - 1
    live = b < case["n_seq"]
    b = b.clamp(max=case["n_seq"] - 1)
    pos = cached[b] + r - row_start[b]
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    wanted = taken.sum()
    counts = torch.stack((wanted.clamp(max=free.numel()), wanted, row_start[-1])).to(torch.int32)
    return {"block_table": table, "slots": torch.where(live, slot, -1), "seq_lens": total.to(torch.int32),
            "row_start": row_start.to(torch.int32), "counts": counts}


def _plain_codec(s, case):
    group, bits = case["group"], case["bits"]
    q, sigma = _quantize(s["x"], s["R"], s["signs"], s["lam"], group, bits)
    slots = s["slots"]
    live = (slots >= 0).nonzero()[:, 0]
    s["codes"][:, slots[live]] = _pack(q, bits)[:, live]
    s["scales"][:, slots[live]] = sigma[:, live]
    x = _dequantize(s["codes"][:, slots[live]], s["scales"][:, slots[live]], s["R"],
                    s["signs"][:, None], s["lam"][:, None], group, bits)
    s["xhat"][:, live] = x.to(torch.float16)
    return s["xhat"]


def _rows_of(table, t, page):
    """Pool rows of the tokens t: table [..., pages] int32, t [tokens]."""
    return table[..., t // page].long().clamp(min=0) * page + t % page


def _plain_attention(s, case):
    H, g, d, page = case["heads"], case["q_per_kv"], case["d"], case["page"]
    B, P, dev = case["n_seq"], case["prefix"], s["q"].device
    how = (case["group"], case["bits"])
    lens = s["seq_lens"].long()
    q = s["q"].to(F32).view(B, H, g, d)
    scale = 1 / math.sqrt(d)
    # the shared tokens once, [H, P, d]; every sequence's own ones, [B, H, T, d]
    tp = torch.arange(P, device=dev)
    T = max(int(_seq_lens(case).max()) - P, 0)
    to = P + torch.arange(T, device=dev)
    rp, ro = _rows_of(s["prefix_table"], tp, page), _rows_of(s["block_table"], to, page)

    def keys(rows):
        return _dequantize(s["k_codes"][rows], s["k_scales"][rows], s["R"], s["sign_k"], s["lam_k"], *how)

    def values(rows):
        return _dequantize(s["v_codes"][rows], s["v_scales"][rows], s["R"], s["sign_v"], s["lam_v"], *how)

    qh = q.permute(1, 0, 2, 3).reshape(H, B * g, d)
    sp = (qh @ keys(rp).permute(1, 2, 0)).view(H, B, g, P).permute(1, 0, 2, 3) * scale
    so = (q @ keys(ro).permute(0, 2, 3, 1)) * scale
    sp = sp.masked_fill((tp >= lens[:, None])[:, None, None], -math.inf)
    so = so.masked_fill((to >= lens[:, None])[:, None, None], -math.inf)
    both = torch.cat((sp, so), -1)
    del sp, so
    top = both.amax(-1, keepdim=True) if P + T else torch.full((B, H, g, 1), -math.inf, device=dev)
    p = torch.exp(both - torch.where(top == -math.inf, 0, top))
    del both
    total = p.sum(-1, keepdim=True)
    pp = p[..., :P].permute(1, 0, 2, 3).reshape(H, B * g, P)
    out = (pp @ values(rp).permute(1, 0, 2)).view(H, B, g, d).permute(1, 0, 2, 3)
    out = out + p[..., P:] @ values(ro).permute(0, 2, 1, 3)
    out = out / torch.where(total > 0, total, 1)
    return out.reshape(B, H * g, d).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _walsh(x):
    shape, d, h = x.shape, x.shape[-1], 1
    while h < d:
        x = x.reshape(-1, d // (2 * h), 2, h)
        x = torch.stack((x[:, :, 0] + x[:, :, 1], x[:, :, 0] - x[:, :, 1]), 2)
        h *= 2
    return x.reshape(shape) / math.sqrt(d)


def _rotate64(u, kind):
    if kind == "srht":
        return _walsh(u)
    d = u.shape[-1]
    X = torch.fft.rfft(u, norm="ortho")
    y = torch.view_as_real(X[..., 1:d // 2]).flatten(-2) * math.sqrt(2)
    return torch.cat((X[..., :1].real, X[..., d // 2:].real, y), -1)


def _unrotate64(y, kind):
    if kind == "srht":
        return _walsh(y)
    d = y.shape[-1]
    mid = torch.view_as_complex(y[..., 2:].reshape(*y.shape[:-1], -1, 2).contiguous()) / math.sqrt(2)
    X = torch.cat((y[..., :1] + 0j, mid, y[..., 1:2] + 0j), -1)
    return torch.fft.irfft(X, n=d, norm="ortho")


def _values64(codes, scales, bits):
    """sigma * code in 64 bits."""
    c = codes.to(torch.int64)
    if bits == 8:
        c = torch.where(c > 127, c - 256, c)
    else:
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        c = torch.where(c > 7, c - 16, c)
    return c.to(F64) * scales.to(F64).repeat_interleave(c.shape[-1] // scales.shape[-1], -1)


def exact(case, seed):
    if case["op"] == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    kind, bits, group = case["rotation"], case["bits"], case["group"]
    if case["op"] == "codec":
        qmax = 2 ** (bits - 1) - 1
        out = s["xhat"].to(F64)
        step = max(1, (1 << 25) // (2 * case["heads"] * case["d"]))
        for a in range(0, case["rows"] - case["padded"], step):
            z = min(a + step, case["rows"] - case["padded"])
            sg, lam = s["signs"][:, None].to(F64), s["lam"][:, None].to(F64)
            w = _rotate64(s["x"][:, a:z].to(F64) * sg, kind) / lam
            w = w.unflatten(-1, (-1, group))
            sigma = (w.abs().amax(-1, keepdim=True) / qmax).clamp(max=65504.0).to(torch.float16).to(F64)
            c = torch.nan_to_num(w / sigma).round().clamp(-qmax, qmax)
            out[:, a:z] = sg * _unrotate64((c * sigma).flatten(-2) * lam, kind)
        return out
    H, g, d, page, P, B = (case[k] for k in ("heads", "q_per_kv", "d", "page", "prefix", "n_seq"))
    lens = s["seq_lens"].tolist()
    longest = max(lens)
    t = torch.arange(max(longest, 1), device=s["q"].device)
    out = torch.zeros((B, H, g, d), dtype=F64, device=t.device)
    top = torch.full((B, H, g), -math.inf, dtype=F64, device=t.device)
    total = torch.zeros((B, H, g), dtype=F64, device=t.device)
    q = s["q"].to(F64).view(B, H, g, d)
    rot_q = _rotate64(q * s["sign_k"][:, None].to(F64), kind) * s["lam_k"][:, None].to(F64) / math.sqrt(d)

    def add(b, rows, h, seen):
        """Tokens of pool rows `rows` for the sequences b (a slice) of head h."""
        k = _values64(s["k_codes"][rows, h], s["k_scales"][rows, h], bits)
        v = _values64(s["v_codes"][rows, h], s["v_scales"][rows, h], bits)
        score = torch.where(seen[:, None, :], rot_q[b, h] @ k.T, -math.inf)
        new = torch.maximum(top[b, h], score.amax(-1))
        fine = torch.where(new == -math.inf, 0, new)
        w, old = torch.exp(score - fine[..., None]), torch.exp(top[b, h] - fine)
        out[b, h] = out[b, h] * old[..., None] + w @ v
        total[b, h] = total[b, h] * old + w.sum(-1)
        top[b, h] = new

    every = s["seq_lens"][:, None]
    for h in range(H):
        for a in range(0, min(P, longest), 16384):
            tt = t[a:min(a + 16384, P, longest)]
            add(slice(0, B), s["prefix_table"][tt // page].long() * page + tt % page, h, tt < every)
        for b in range(B):
            if lens[b] > P:
                tt = t[P:lens[b]]
                rows = s["block_table"][b, tt // page].long() * page + tt % page
                add(slice(b, b + 1), rows, h, torch.ones_like(tt, dtype=torch.bool)[None])
    y = out / torch.where(total > 0, total, 1)[..., None] * s["lam_v"][:, None].to(F64)
    return (_unrotate64(y, kind) * s["sign_v"][:, None].to(F64)).reshape(B, H * g, d)
