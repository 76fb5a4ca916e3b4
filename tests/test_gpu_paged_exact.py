"""fp16 outputs of the shared-prefix attention to the precision that their split
operands give (paged_exact), on every kernel that has the split."""

import math

import numpy as np
import pytest

import rotate_then_quantize_b200 as rq

import paged
import paged_exact
from test_gpu_paged import _attn_case, _ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gain,slack", [(1.0, paged_exact.TIGHT), (5.0, paged_exact.PEAKED)])
@pytest.mark.parametrize("n_seq,prefix", [(3, 0), (5, 400), (20, 6600)])
@pytest.mark.parametrize("d,bits,group,rot", [
    (64, 4, 16, 0), (64, 8, 32, 1), (128, 4, 16, 0), (128, 8, 16, 1), (128, 4, 128, 0),
    (256, 4, 32, 0), (256, 8, 16, 1)])
def test_fp16_outputs(n_seq, prefix, d, bits, group, rot, gain, slack):
    """Own tokens, a short prefix by warp-level tiles, a long one by tcgen05."""
    rng = np.random.default_rng(n_seq + d + bits + group)
    g = 8 if d == 256 else 4
    own = _ragged(rng, n_seq, 900 if prefix == 0 else 200)
    q, dev, host = _attn_case(rng, n_seq, 2, g, d, bits, group, rot, prefix, own, 16, "float16",
                              q_gain=gain)
    host["vhat"] = paged_exact.rounded_values(
        dev["v_codes"].cpu().numpy(), dev["v_scales"].cpu().numpy(), dev["v_signs"].cpu().numpy(),
        dev["v_lambda"].cpu().numpy(), bits, group, rot)
    out = rq.prefix_attention(q, **dev).double().cpu().numpy()
    assert rq.srftq_check_device() == 0
    ref, _ = paged.attention(q.double().cpu().numpy(), scale=1 / math.sqrt(d), **host)
    assert paged_exact.worst(out, ref, slack) <= 1.0
