"""The shared-prefix attention over the whole range of the scales, on each of its
kernels: scales so small that they are subnormal fp16 numbers, and so large that a
scale times a code passes fp16's end. Both sides take the same codes and scales,
lambda making up for the scales' size, so the bound is that of
paged.check_attention, which counts a rounding of each product to 11 bits."""

import numpy as np
import pytest

import oracle
import rotate_then_quantize_b200 as rq

import paged
from test_gpu_paged import DEV, _attn_case, _check, _ragged, _t

pytestmark = pytest.mark.gpu


def _rescale(q, dev, host, factor, lam, which="kv"):
    """Scales times `factor` (an array over the pool's rows, or a number), rounded
    to fp16, lambda times `lam`; the host's vectors from what the device gets."""
    bits, group, d, rot = dev["bits"], dev["group"], q.shape[2], dev["rotation"]
    for c in which:
        s = dev[c + "_scales"].double().cpu().numpy()
        s = (s * np.reshape(factor, (-1, 1, 1))).astype(np.float16)
        assert np.isfinite(s).all()
        dev[c + "_scales"] = _t(s)
        dev[c + "_lambda"] = dev[c + "_lambda"] * lam
        host[c + "hat"] = oracle.dequantize(
            dev[c + "_codes"].cpu().numpy()[None], s.view(np.uint16)[None],
            dev[c + "_signs"].cpu().numpy()[None], dev[c + "_lambda"].cpu().numpy()[None], d, group,
            bits, rot)["xhat64"][0]


KERNELS = [   # n_seq, prefix, d, dtype: warp-level tiles; two units, the same rows, other rows; one unit
    (3, 100, 128, "float16"), (3, 100, 64, "bfloat16"), (20, 6600, 128, "float16"),
    (20, 6600, 64, "bfloat16"), (50, 6600, 128, "bfloat16"), (50, 6600, 64, "bfloat16"),
    (30, 6600, 256, "float16"), (30, 6600, 256, "bfloat16")]


def _case(n_seq, prefix, d, dtype, bits, group=16, seed=0):
    rng = np.random.default_rng(n_seq + bits + d + seed)
    return rng, *_attn_case(rng, n_seq, 2, 4, d, bits, group, 0, prefix, _ragged(rng, n_seq, 90), 16,
                            dtype)


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS)
@pytest.mark.parametrize("bits,k", [(8, 9), (8, 12), (4, 13), (4, 16)])
def test_subnormal_scales(n_seq, prefix, d, dtype, bits, k):
    """Scales around 2^-15 and 2^-18, lambda 2^k times as large."""
    _, q, dev, host = _case(n_seq, prefix, d, dtype, bits)
    _rescale(q, dev, host, 2.0 ** -k, 2.0 ** k)
    small = dev["v_scales"].float()
    assert float(small.median()) < 2.0 ** -14 and float(small.max()) > 0
    _check(q, dev, host)


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("which", ["k", "v"])
def test_large_scales(n_seq, prefix, d, dtype, bits, which):
    """Some tokens with scales past 8192 (int4) or 512 (int8), among shared and own
    ones; lambda as much smaller, so that scores and outputs are of order one."""
    rng, q, dev, host = _case(n_seq, prefix, d, dtype, bits, group=32, seed=5)
    up = 2.0 ** 15
    factor = np.ones(dev["k_codes"].shape[0])
    pt, table = host["prefix_table"], host["block_table"]
    factor[paged.rows_of(pt, np.array([7, prefix // 2, prefix - 1]), 16, 10 ** 9)] = up
    factor[paged.rows_of(table[0], prefix + np.array([0, 40, 85]), 16, 10 ** 9)] = up
    _rescale(q, dev, host, factor, 2.0 / up, which)
    limit = 8192 if bits == 4 else 512
    assert float(dev[which + "_scales"].max()) >= limit
    _check(q, dev, host)


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS)
def test_every_scale_at_the_end_of_fp16(n_seq, prefix, d, dtype):
    """The codec's largest scale, 65504, in every token of keys and values."""
    _, q, dev, host = _case(n_seq, prefix, d, dtype, 8)
    for c in "kv":
        dev[c + "_scales"].fill_(65504.0)
    _rescale(q, dev, host, 1.0, 2.0 ** -21)
    _check(q, dev, host)


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS)
def test_large_and_non_finite_scales(n_seq, prefix, d, dtype):
    """A scale that is not finite keeps to the sequences that attend to its token
    when others are large; the rest is right."""
    import torch
    _, q, dev, host = _case(n_seq, prefix, d, dtype, 4, seed=9)
    lens = host["seq_lens"]
    lens[1], lens[2] = prefix // 2, prefix // 2 + 1
    dev["seq_lens"] = _t(lens.astype(np.int32))
    factor = np.ones(dev["k_codes"].shape[0])
    row = lambda t: int(paged.rows_of(host["prefix_table"], np.array([t]), 16, 10 ** 9)[0])
    factor[row(3)] = 2.0 ** 15
    _rescale(q, dev, host, factor, 2.0 ** -12, "v")
    dev["v_scales"][row(prefix // 2), 1, 0] = float("nan")
    out = rq.prefix_attention(q, **dev)
    assert rq.srftq_check_device() == 0
    hit = _t(lens > prefix // 2)
    assert not bool(out[hit][:, 4:].isfinite().any())
    ref, _ = paged.attention(q.double().cpu().numpy(), scale=d ** -0.5, **host)
    for part in (out[:, :4], out[~hit]):
        assert bool(part.isfinite().all())
    got = out.double().cpu().numpy()
    got[(lens > prefix // 2)[:, None] & (np.arange(8) >= 4)] = 0
    ref[(lens > prefix // 2)[:, None] & (np.arange(8) >= 4)] = 0
    paged.check_attention(got, ref, torch.finfo(q.dtype).eps)


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS)
def test_nothing_stays_from_a_call_with_large_scales(n_seq, prefix, d, dtype):
    """Calls with and without large scales in turn, in one workspace, eager and
    captured: the result each has by itself."""
    import torch
    _, q, dev, host = _case(n_seq, prefix, d, dtype, 4, seed=2)
    want = [rq.prefix_attention(q, **dev)]
    large = dict(dev)
    large["v_scales"] = dev["v_scales"].clone()
    large["v_scales"][int(host["prefix_table"][0]) * 16] = 20000.0
    large["v_lambda"] = dev["v_lambda"] * 2.0 ** -12
    want.append(rq.prefix_attention(q, **large))
    need = rq.srftq_prefix_attention_workspace(rq.make_desc(d, 2, 16, 4), n_seq, 4, prefix)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for i, x in enumerate((dev, large)):
            assert torch.equal(rq.prefix_attention(q, **x, workspace=ws), want[i])
    out = torch.empty_like(q)
    scales, lam = dev["v_scales"].clone(), dev["v_lambda"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq.prefix_attention(q, **{**dev, "v_scales": scales, "v_lambda": lam}, workspace=ws, out=out)
    for i, x in enumerate((large, dev, large)):
        scales.copy_(x["v_scales"])
        lam.copy_(x["v_lambda"])
        graph.replay()
        assert torch.equal(out, want[(1, 0, 1)[i]])


@pytest.mark.parametrize("n_seq,prefix,d,dtype", KERNELS + [(40, 0, 128, "float16"),
                                                            (40, 0, 64, "bfloat16")])
@pytest.mark.parametrize("bits,group", [(4, 16), (8, 64)])
def test_infinite_key_scale(n_seq, prefix, d, dtype, bits, group):
    """An infinite scale of keys makes NaN of every query head that attends to its
    token, whatever the signs of its codes and query; a score of -inf would leave
    the token out without a word."""
    _, q, dev, host = _case(n_seq, prefix, d, dtype, bits, group, seed=7)
    want = rq.prefix_attention(q, **dev)
    table, t = (host["prefix_table"], 3) if prefix else (host["block_table"][0], 3)
    row = int(paged.rows_of(table, np.array([t]), 16, 10 ** 9)[0])
    ng = d // group
    for g, value in ((0, np.inf), (ng - 1, -np.inf)):
        scales = dev["k_scales"].clone()
        scales[row, 1, g] = value
        got = rq.prefix_attention(q, **{**dev, "k_scales": scales})
        hit = _t(host["seq_lens"] > t) if prefix else _t(np.arange(n_seq) == 0)
        assert bool(got[hit][:, 4:].isnan().all())
        assert bool((got[:, :4] == want[:, :4]).all()) and bool((got[~hit] == want[~hit]).all())
    assert rq.srftq_check_device() == 0
