"""The paged calls on the debug build, whose kernels check every index that they
compute: no check fails, and the results are those of the release build."""

import os

import numpy as np
import pytest

import rotate_then_quantize_b200 as rq
from rotate_then_quantize_b200 import binding as b

from test_gpu_paged import DEV, _attn_case, _ragged, _t, _tables_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _debug_library():
    if not os.path.exists(b.LIB_DEBUG_PATH):
        from rotate_then_quantize_b200 import build
        build.build(debug=True)
    rq.load_library(b.LIB_DEBUG_PATH)


def _both(call):
    """The results of `call` on either build; the debug build's checks are silent."""
    want = call()
    with rq.debug_checks():
        assert rq.srftq_debug_checks() and rq.srftq_check_device() == 0
        got = call()
        assert rq.srftq_check_device() == 0
    import torch
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n_seq,page,short,narrow,pad", [(1, 16, 0, 0, 0), (40, 16, 11, 5, 4),
                                                         (2100, 7, 0, 0, 3000), (33, 24, 0, 0, -50)])
def test_tables_under_index_checks(n_seq, page, short, narrow, pad):
    rng = np.random.default_rng(n_seq)
    c, n, table, free, total = _tables_case(rng, n_seq, page, 90, 60, short, narrow)

    def call():
        t = _t(table)
        return (t, *rq.block_tables(_t(c.astype(np.int32)), _t(n.astype(np.int32)), _t(free), t, page,
                                    max(total + pad, 0)))
    _both(call)


@pytest.mark.parametrize("d,bits,group", [(64, 4, 16), (128, 8, 128), (128, 4, 16), (256, 4, 32),
                                          (256, 8, 16)])
@pytest.mark.parametrize("N,H", [(1, 1), (77, 3), (400, 8)])
def test_codec_under_index_checks(d, bits, group, N, H):
    import torch
    rng = np.random.default_rng(N + d)
    rows = N + 9
    x = _t(rng.standard_normal((2, N, H, d)).astype(np.float16))
    signs = _t(np.where(rng.random((2, H, d)) < 0.5, -1, 1).astype(np.int8))
    lam = torch.rand((2, H, d), device=DEV) + 0.5
    slots = rng.permutation(rows)[:N].astype(np.int64)
    slots[rng.random(N) < 0.2] = -1
    slots[0] = rows + (1 << 40)
    slots = _t(slots)

    def call():
        codes = torch.zeros((2, rows, H, d * bits // 8), dtype=torch.uint8, device=DEV)
        scales = torch.zeros((2, rows, H, d // group), dtype=torch.float16, device=DEV)
        rq.quantize_paged(x, signs, lam, slots, codes, scales, group, bits)
        return codes, scales, rq.dequantize_paged(codes, scales, slots, signs, lam, d, group, bits)
    _both(call)


@pytest.mark.parametrize("d,bits,group,dtype", [(64, 4, 16, "float16"), (128, 8, 16, "bfloat16"),
                                                (128, 4, 128, "float16"), (256, 4, 32, "bfloat16")])
@pytest.mark.parametrize("n_seq,g,prefix,page", [(1, 1, 0, 1), (5, 3, 100, 24), (70, 4, 7001, 16),
                                                 (20, 8, 7001, 7), (330, 8, 65, 16)])
def test_attention_under_index_checks(d, bits, group, dtype, n_seq, g, prefix, page):
    """Tiles, both tcgen05 kernels, each form of the join; bad pages, empty and short
    sequences, a large scale and one that is not finite."""
    rng = np.random.default_rng(n_seq + d)
    own = _ragged(rng, n_seq, 40)
    if n_seq > 3:
        own[1], own[2] = -1, -1 - prefix // 2
    q, dev, host = _attn_case(rng, n_seq, 2, g, d, bits, group, 0, prefix, own, page, dtype)
    dev["block_table"][0, 0] = 2 ** 31 - 1
    _both(lambda: rq.prefix_attention(q, **dev, return_lse=True))
    if prefix:
        row = int(host["prefix_table"][0]) * page
        dev["v_scales"][row] = 20000.0
        _both(lambda: rq.prefix_attention(q, **dev, return_lse=True))
        dev["k_scales"][row, 1] = float("inf")
        dev["seq_lens"][:2] = 0
        _both(lambda: [x.nan_to_num() for x in rq.prefix_attention(q, **dev, return_lse=True)])
