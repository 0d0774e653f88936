"""FP4 E2M1 cache codec (oracle; test infrastructure only).

The 4-bit form of the quantised latent cache of [CF] "Smaller, faster, safer: running
Kimi and GLM at scale", section "Quantizing the KV cache". The page names no 4-bit
format; the readings are ours:

* an element is an OCP E2M1 code: 1 sign bit, 2 exponent bits with bias 1, 1 mantissa
  bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; no NaN and no infinity;
* 32 consecutive elements of an entry share a power of two 2^e, -8 <= e <= 6, stored as
  the nibble n = e + 8; n = 15 marks a block that held a NaN and reads as NaN;
* value = e2m1 * 2^e * kv_scale.

Write side: e is the smallest power with max|x| <= 7 * 2^e * kv_scale (6 if none), and the
code is the nearest magnitude to |x| / (2^e * kv_scale), the even code on a tie, 6 above.

A page of 64 tokens is 19,008 bytes: codes [18][64][16] (block, token, bytes; the even
element in the low nibble), then exponents [9][64] (byte i: block 2i low, 2i + 1 high).
"""

from __future__ import annotations

import numpy as np

PAGE = 64
ENTRY = 576
BLOCK = 32
BLOCKS = ENTRY // BLOCK
CODE_BYTES = BLOCKS * PAGE * 16
PAGE_BYTES = CODE_BYTES + (BLOCKS // 2) * PAGE
NAN_EXP = 15


def code_value(code: int) -> float:
    """Value of one e2m1 code, written straight from the format definition."""
    exp, mant = (code >> 1) & 3, code & 1
    mag = 0.5 * mant if exp == 0 else (1.0 + 0.5 * mant) * 2.0 ** (exp - 1)
    return -mag if code & 8 else mag


MAGNITUDES = np.array([code_value(c) for c in range(8)])


def encode(x: np.ndarray, kv_scale: float):
    """Codes ``[..., 576]`` (0..15) and nibbles ``[..., 18]`` of exact entries ``x [..., 576]``.

    float64 throughout: products of a 3-bit midpoint, a 24-bit scale and a power of two
    are exact, so no comparison is affected by rounding.
    """
    x = np.asarray(x, dtype=np.float64)
    scale = np.float64(np.float32(kv_scale))
    blk = x.reshape(*x.shape[:-1], BLOCKS, BLOCK)
    amax = np.abs(blk).max(axis=-1)
    nan = np.isnan(blk).any(axis=-1)
    exp = np.full(amax.shape, 6, dtype=np.int64)
    for e in range(5, -9, -1):
        with np.errstate(invalid="ignore"):
            exp = np.where(amax <= 7.0 * 2.0 ** e * scale, e, exp)
    unit = np.ldexp(scale, exp)[..., None]
    codes = np.zeros(blk.shape, dtype=np.int64)
    for c in range(7):
        mid = (MAGNITUDES[c] + MAGNITUDES[c + 1]) / 2.0 * unit
        with np.errstate(invalid="ignore"):
            up = np.abs(blk) >= mid if (c + 1) % 2 == 0 else np.abs(blk) > mid
        codes += up
    codes |= np.where(np.signbit(blk), 8, 0)
    codes = np.where(nan[..., None], 0, codes)
    nibs = np.where(nan, NAN_EXP, exp + 8)
    return codes.reshape(x.shape).astype(np.uint8), nibs.astype(np.uint8)


def values(codes: np.ndarray, nibs: np.ndarray, kv_scale: float) -> np.ndarray:
    """Entries ``[..., 576]`` in float64 of codes and nibbles as :func:`encode` gives them."""
    table = np.array([code_value(c) for c in range(16)])
    power = np.ldexp(1.0, np.arange(16) - 8)
    power[NAN_EXP] = np.nan
    return table[codes] * np.repeat(power[nibs], BLOCK, axis=-1) * np.float64(np.float32(kv_scale))


def store(pages: np.ndarray, slots: np.ndarray, codes: np.ndarray, nibs: np.ndarray) -> None:
    """Writes tokens' codes and nibbles into ``pages [num_pages, 19008]`` at their slots, in place."""
    for slot, c, n in zip(np.asarray(slots).tolist(), codes, nibs):
        if slot < 0 or slot >= pages.shape[0] * PAGE:
            continue
        page, t = pages[slot // PAGE], slot % PAGE
        page[:CODE_BYTES].reshape(BLOCKS, PAGE, 16)[:, t] = (c[0::2] | (c[1::2] << 4)).reshape(BLOCKS, 16)
        page[CODE_BYTES:].reshape(BLOCKS // 2, PAGE)[:, t] = n[0::2] | (n[1::2] << 4)


def load(pages: np.ndarray):
    """Codes ``[num_pages, 64, 576]`` and nibbles ``[num_pages, 64, 18]`` of stored pages."""
    n = pages.shape[0]
    raw = pages[:, :CODE_BYTES].reshape(n, BLOCKS, PAGE, 16).transpose(0, 2, 1, 3).reshape(n, PAGE, ENTRY // 2)
    exps = pages[:, CODE_BYTES:].reshape(n, BLOCKS // 2, PAGE).transpose(0, 2, 1)
    codes = np.stack([raw & 15, raw >> 4], axis=-1).reshape(n, PAGE, ENTRY)
    nibs = np.stack([exps & 15, exps >> 4], axis=-1).reshape(n, PAGE, BLOCKS)
    return codes, nibs


def decode_pages(pages: np.ndarray, kv_scale: float) -> np.ndarray:
    """Entries ``[num_pages, 64, 576]`` in float64 of stored pages."""
    return values(*load(pages), kv_scale)
