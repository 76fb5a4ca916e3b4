"""That the bound of paged_exact holds for the arithmetic as it is meant and fails
for one without any one of its rests (numpy, no GPU)."""

import numpy as np
import pytest

import oracle

import paged
import paged_exact


@pytest.mark.parametrize("gain,slack", [(1.0, paged_exact.TIGHT), (5.0, paged_exact.PEAKED)])
@pytest.mark.parametrize("d,bits,group,rot", [(64, 4, 16, 0), (128, 8, 16, 1), (128, 4, 64, 0),
                                              (256, 4, 32, 0), (256, 8, 256, 1)])
def test_a_lost_rest_fails_the_bound(d, bits, group, rot, gain, slack):
    rng = np.random.default_rng(d + bits + group)
    tokens, rows = 1500, 24
    kc, ks, ksg, kl, kh = paged.cache(rng, tokens, 1, d, bits, group, rot)
    vc, vs, vsg, vl, _ = paged.cache(rng, tokens, 1, d, bits, group, rot)
    q = (gain * rng.standard_normal((rows, d))).astype(np.float16)
    vh = paged_exact.rounded_values(vc, vs, vsg, vl, bits, group, rot)
    s = q.astype(np.float64) @ kh[:, 0].T / np.sqrt(d)
    p = np.exp(s - s.max(-1, keepdims=True))
    ref = p @ vh[:, 0] / p.sum(-1, keepdims=True)

    def products(codes, scales):
        c = oracle.unpack_codes(codes, bits)[:, 0].astype(np.float64)
        return c * np.repeat(scales.view(np.float16)[:, 0].astype(np.float64), group, -1)

    def ratio(lost):
        out = paged_exact.model(q.astype(np.float64), products(kc, ks), products(vc, vs), kl[0],
                                vl[0], ksg[0], vsg[0], rot, lost)
        return paged_exact.worst(out, ref, slack)

    assert ratio(None) <= 1.0
    for lost in ("query", "keys") if gain > 1 else ("query", "keys", "weights"):
        assert ratio(lost) > 1.0, lost
