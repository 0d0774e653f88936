"""The 4-bit codec oracle is pinned by the format definition, exact arithmetic and torch (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import e2m1 as o
from oracle import e4m3

SCALES = [float(np.float32(s)) for s in (4.0 / 448.0, 1.0, 0.1, 2.0 ** -100, 2.0 ** 100)]


def test_code_values():
    assert [o.code_value(c) for c in range(8)] == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert [o.code_value(c) for c in range(8, 16)] == [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def test_every_stored_value_is_an_e4m3_number():
    """The exponents -8 .. 6 are those for which the 4-bit values are e4m3 values."""
    grid = set(e4m3.DECODE_TABLE[~np.isnan(e4m3.DECODE_TABLE)].tolist())
    for n in range(15):
        for c in range(16):
            assert o.code_value(c) * 2.0 ** (n - 8) in grid
    assert 6.0 * 2.0 ** 7 not in grid and 0.5 * 2.0 ** -9 not in grid


@pytest.mark.parametrize("scale", SCALES)
def test_encode_is_the_nearest_value_in_exact_arithmetic(scale):
    """Against rationals: the smallest admissible power, then the nearest magnitude, ties to even."""
    rng = np.random.default_rng(3)
    x = np.ldexp(rng.integers(-255, 256, (40, 576)).astype(np.float64), rng.integers(-20, 8, (40, 576))) * scale
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    x = e4m3.bf16_bits_to_f64(bits)
    x[0, :32] = 0.0
    codes, nibs = o.encode(x, scale)
    s = Fraction(scale)
    for i in range(x.shape[0]):
        for b in range(18):
            blk = [Fraction(v) for v in x[i, 32 * b:32 * b + 32]]
            top = max(abs(v) for v in blk)
            e = next((e for e in range(-8, 6) if top <= 7 * s * Fraction(2) ** e), 6)
            assert nibs[i, b] == e + 8
            for k in range(0, 32, 5):
                q = abs(blk[k]) / (s * Fraction(2) ** e)
                far = [abs(q - Fraction(m)) for m in o.MAGNITUDES]
                best = min(range(8), key=lambda c: (far[c], c % 2))
                assert codes[i, 32 * b + k] % 8 == best


def test_signs_infinities_and_nans():
    x = np.zeros((3, 576))
    x[0, 0], x[0, 1] = -0.0, np.inf
    x[1, 5], x[1, 6] = np.nan, 3.0
    x[2, 40] = -np.inf
    codes, nibs = o.encode(x, 1.0)
    v = o.values(codes, nibs, 1.0)
    assert codes[0, 0] == 8 and v[0, 1] == 384.0 and nibs[0, 0] == 14
    assert np.isnan(v[1, :32]).all() and (codes[1, :32] == 0).all() and (v[1, 32:] == 0).all()
    assert v[2, 40] == -384.0 and not np.isnan(v[2]).any()


def test_rounding_error_is_at_most_a_sixth_of_the_blocks_largest():
    """Between 4 and 6 units the half step is 1; blocks are scaled so that the largest
    magnitude lies above 3.5 units (and up to 7, which is 1 above the last value)."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((200, 576))
    v = o.values(*o.encode(x, 4.0 / 448.0), 4.0 / 448.0)
    err = np.abs(v - x).reshape(200, 18, 32)
    top = np.abs(x).reshape(200, 18, 32).max(-1, keepdims=True)
    assert (err <= top / 3.5 + 1e-12).all()
    assert (err.max(-1) <= top[..., 0] * (1.0 / 3.5) + 1e-12).all()


def test_store_and_load_are_inverse():
    rng = np.random.default_rng(7)
    codes = rng.integers(0, 16, (200, 576)).astype(np.uint8)
    nibs = rng.integers(0, 16, (200, 18)).astype(np.uint8)
    slots = rng.permutation(5 * 64)[:200]
    pages = np.full((5, o.PAGE_BYTES), 0xAA, dtype=np.uint8)
    o.store(pages, slots, codes, nibs)
    c, n = o.load(pages)
    assert np.array_equal(c.reshape(-1, 576)[slots], codes)
    assert np.array_equal(n.reshape(-1, 18)[slots], nibs)
    rest = np.setdiff1d(np.arange(320), slots)
    assert (c.reshape(-1, 576)[rest] == 0xA).all() and (n.reshape(-1, 18)[rest] == 0xA).all()
    assert o.PAGE_BYTES == 19008
