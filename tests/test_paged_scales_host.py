"""The fp16 products of scales and codes that the shared-prefix attention holds
(csrc/paged_attention.cuh, prefix_mma.cuh), restated in numpy: every scale below
the large ones keeps eleven bits of every product, the smallest subnormals too,
and the decoding from fp16 bit patterns is exact."""

import re
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rotate_then_quantize_b200", "csrc")


def _half(bits):
    return np.array(bits, np.uint16).view(np.float16).astype(np.float64)


@pytest.mark.parametrize("bits", [4, 8])
def test_products_keep_eleven_bits(bits):
    text = open(os.path.join(CSRC, "paged_attention.cuh")).read()
    m = re.search(r"kLargeScale = BITS == 4 \? 0x(\w+)u : 0x(\w+)u", text)
    large = int(m.group(1 if bits == 4 else 2), 16)
    most = 8 if bits == 4 else 128
    scales = _half(np.arange(large))                 # every scale below the large ones
    assert _half(large) == {4: 8192, 8: 512}[bits]
    for c in range(1, most + 1):
        exact = scales * c
        held = exact.astype(np.float16)
        assert np.isfinite(held).all()
        assert (np.abs(held.astype(np.float64) - exact) <= 2.0 ** -11 * exact).all()
        # what the rounding left, for fp16 outputs' keys: exact too
        rest = exact - held.astype(np.float64)
        assert (rest.astype(np.float16).astype(np.float64) == rest).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_large_halves(bits):
    """The packed test for large scales, over every pair of a pattern and a few."""
    large = 0x7000 if bits == 4 else 0x6000
    lo = np.arange(65536, dtype=np.uint64)
    for hi in (0, 1, large - 1, large, 0x7C00, 0x7FFF, 0x8000, 0x8000 + large - 1, 0xFFFF):
        s = lo | (np.uint64(hi) << np.uint64(16))
        got = (((s & np.uint64(0x7FFF7FFF)) + np.uint64((0x8000 - large) * 0x10001))
               & np.uint64(0x80008000))
        assert ((got & np.uint64(0x8000) != 0) == ((lo & np.uint64(0x7FFF)) >= large)).all()
        assert ((got >> np.uint64(31) != 0) == ((hi & 0x7FFF) >= large)).all()


def test_decoding_is_exact():
    """1024 + u and 1024 + 16 u, times a power of two, plus a constant: the code."""
    u = np.arange(16)
    low = _half(0x6400 + u) * _half(0x3C00) + _half(0xE408)
    high = _half(0x6400 + 16 * u) * _half(0x2C00) + _half(0xD480)
    assert (low == u - 8).all() and (high == u - 8).all()
    u = np.arange(256)
    assert (_half(0x6400 + u) * _half(0x3C00) + _half(0xE480) == u - 128).all()
