// kv_e2m1.cuh -- the 4-bit cache format (MLA_KV_E2M1): page layout, the rounding
// thresholds of the write side and the expansion tables of the read side.
//
// A page of 64 tokens is 19,008 contiguous bytes:
//   codes [18 blocks][64 tokens][16 B]  block b of a token = its elements 32b .. 32b+31,
//                                       two e2m1 codes per byte, the even element low
//   exps  [9][64 tokens]                byte i: blocks 2i (low nibble) and 2i+1 (high)
// value = e2m1(code) * 2^(n - 8) * kv_scale with n the block's nibble; n = 15: NaN.
// Codes of one block lie beside each other for consecutive tokens, so that eight
// threads with consecutive tokens read 128 contiguous bytes and write eight rows of a
// swizzled tensor-core operand without bank conflicts (decode_fp8.cu).
//
// The exponents 2^-8 .. 2^6 are those for which every e2m1 value times the power is an
// e4m3 number (0.5 * 2^-8 = 2^-9, the smallest; 6 * 2^6 = 384 <= 448): a 4-bit page
// expands to e4m3 codes exactly, and the tensor-core path of the e4m3 cache applies.
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "mla_common.cuh"

namespace mla {

constexpr int kE2m1Block = MLA_E2M1_BLOCK;                  // 32 elements share an exponent
constexpr int kE2m1Blocks = kDEntry / kE2m1Block;           // 18
constexpr int kE2m1CodeBytes = kE2m1Blocks * kPageSize * 16;  // 18,432
constexpr int kE2m1PageBytes = MLA_E2M1_PAGE_BYTES;         // 19,008
constexpr int kE2m1NanExp = 15;
static_assert(kE2m1CodeBytes + kE2m1Blocks / 2 * kPageSize == kE2m1PageBytes, "page layout");

// Byte offset within a page of the 16 code bytes of (block, token), and of the exponent
// byte that holds the block's nibble.
__host__ __device__ constexpr int e2m1_code_offset(int block, int token) {
  return (block * kPageSize + token) * 16;
}
__host__ __device__ constexpr int e2m1_exp_offset(int block, int token) {
  return kE2m1CodeBytes + (block >> 1) * kPageSize + token;
}

// ---- write side ----
// Thresholds as float32 for scale s, such that for every float32 y:
//   y >= step[i]  <=>  |x| = y (already divided by 2^e) rounds above e2m1 value i, i.e.
//                      y is beyond the midpoint of values i and i + 1 times s, or on it
//                      when the even code is i + 1;
//   amax <= top * 2^e  <=>  amax <= 7 * s * 2^e.
// The products (27 significant bits at most) are formed exactly in double; the nearest
// float32 on the right side of each decides every float32 y as the product would.
// s must lie in [2^-100, 2^100], so that no threshold over- or underflows.
//
// `inverse` (0 if there is none): a float32 r for which the hardware's rounding of
// fl(y * r) to e2m1 agrees with the thresholds for every bf16 y. A product is rounded to
// 24 bits, so this is a property of the bf16 numbers on either side of each threshold,
// checked here for 1/s and its neighbours up to two units away. Of the 2^23 mantissas of
// s only 1.875 has none (its midpoints are exact ties of bf16 numbers, and no r hits all).
struct E2m1Steps {
  float step[7];
  float top;
  float inverse;
};
inline float e2m1_round_down(double d) {
  const float f = (float)d;
  return (double)f > d ? nextafterf(f, -INFINITY) : f;
}
inline float e2m1_round_up(double d) {
  const float f = (float)d;
  return (double)f < d ? nextafterf(f, INFINITY) : f;
}
inline E2m1Steps e2m1_steps(float s) {
  const float mid[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
  E2m1Steps r;
  float above[7], below[7];  // the bf16 numbers on either side of each threshold
  for (int i = 0; i < 7; ++i) {
    const double t = (double)mid[i] * (double)s;
    r.step[i] = (i & 1) ? e2m1_round_up(t) : nextafterf(e2m1_round_down(t), INFINITY);
    uint32_t bits;
    memcpy(&bits, &r.step[i], 4);
    bits = (bits + 0xffffu) & 0xffff0000u;
    memcpy(&above[i], &bits, 4);
    bits -= 0x10000u;
    memcpy(&below[i], &bits, 4);
  }
  r.top = e2m1_round_down(7.0 * (double)s);
  r.inverse = 0.f;
  for (int k = 0; k < 5 && r.inverse == 0.f; ++k) {
    float c = 1.0f / s;
    for (int n = 0; n < (k + 1) / 2; ++n) c = nextafterf(c, (k & 1) ? INFINITY : 0.f);
    bool ok = true;
    for (int i = 0; i < 7; ++i) {
      const float a = above[i] * c, b = below[i] * c;
      ok = ok && ((i & 1) ? a >= mid[i] && b < mid[i] : a > mid[i] && b <= mid[i]);
    }
    if (ok) r.inverse = c;
  }
  return r;
}
inline bool e2m1_scale_ok(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

// ---- read side ----
// e4m3 codes of the eight magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^(n - 8), one byte
// each, magnitude 0 in the lowest byte; 0x7f (NaN) throughout for n = 15.
__host__ __device__ constexpr uint64_t e2m1_as_e4m3(int n) {
  const int halves[8] = {0, 1, 2, 3, 4, 6, 8, 12};  // the magnitudes in units of 0.5
  uint64_t row = 0;
  for (int c = 0; c < 8; ++c) {
    uint64_t code = 0;
    const int v = halves[c];
    if (n == kE2m1NanExp) {
      code = 0x7f;
    } else if (v > 0) {
      int k = 0;
      while ((v >> (k + 1)) > 0) ++k;     // v = (1 + m/2) * 2^k
      const int m = v == (1 << k) ? 0 : 1;
      const int e = k + n - 9;            // value = (1 + m/2) * 2^e
      code = e >= -6 ? (uint64_t)(((e + 7) << 3) | (m << 2)) : (uint64_t)(v << n);
    }
    row |= code << (8 * c);
  }
  return row;
}

// Eight e2m1 codes (nibble i = element i) -> eight e4m3 codes, given the block's table
// row (lo: magnitudes 0..3, hi: 4..7): nine instructions. A byte permute looks up four
// magnitudes at once; the signs are the top bits of w's bytes (odd elements) and of
// w << 4 (even elements), which another permute puts in element order.
__device__ __forceinline__ uint2 e2m1x8_to_e4m3(uint32_t w, uint32_t lo, uint32_t hi) {
  const uint32_t mag = w & 0x77777777u, even = w << 4;
  const uint32_t s0 = __byte_perm(even, w, 0x5140), s1 = __byte_perm(even, w, 0x7362);
  return make_uint2(__byte_perm(lo, hi, mag) | (s0 & 0x80808080u),
                    __byte_perm(lo, hi, mag >> 16) | (s1 & 0x80808080u));
}

}  // namespace mla
