// prob_rows.cuh -- rows of probabilities as exact integer weights, and wide loads of rows.
//
// Shared by the verifications of drafts (verify_drafts.cu, verify_tree.cu): a probability
// becomes an integer in units of 2^-60, so that sums are exact and do not depend on the
// order of addition.
#pragma once

#include "mla_common.cuh"

namespace mla {
namespace {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// A probability within [0, 1] (NaN and negative values: 0).
__device__ __forceinline__ float weight(float x) { return __saturatef(x); }
// weight(x) in units of 2^-60 as three slices of 20 bits, s[0] 2^40 + s[1] 2^20 + s[2].
// Adding 8 to x leaves x rounded to 2^-20 in the low bits of the float32 sum; what the
// rounding left over is exact, and 1.5 * 2^-17 and 1.5 * 2^-37 do the same for it with
// 2^-40 and 2^-60 (signed: the low bits of a sum count from those of its constant, so the
// slices of a difference are differences of the sums as integers). Six additions on the
// full-rate pipe per number. For 128 requests of 163,840 tokens conversions to a 64-bit
// integer took 84 us, shifts by the exponent 41, this 36 (122 MB read).
struct Slices {
  int32_t s[3];
};
__device__ __forceinline__ Slices slices(float w) {
  constexpr float kA = 8.f, kB = 0x1.8p-17f, kC = 0x1.8p-37f;
  constexpr float kBC = kB + kC;  // exact: 21 bits
  Slices r;
  const float a = w + kA;
  const float rest = w - (a - kA);
  const float b = rest + kB;
  r.s[0] = __float_as_int(a);
  r.s[1] = __float_as_int(b);
  r.s[2] = __float_as_int(rest - (b - kBC));  // (rest - slice 1) + kC, rounded once
  return r;
}
__device__ __forceinline__ uint64_t joined(const Slices& w) {
  return ((uint64_t)(int64_t)w.s[0] << 40) + ((uint64_t)(int64_t)w.s[1] << 20) +
         (uint64_t)(int64_t)w.s[2];
}
__device__ __forceinline__ float unit(float u) { return u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f; }
// floor(u * total) for a uniform u, which from 2^-41 on is a multiple of 2^-64; a smaller one is
// first raised by a power of two (as exact as the rest, and no time where there is none).
__device__ __forceinline__ uint64_t share(float u, uint64_t total) {
  int shift = 0;
  while (__builtin_expect(u > 0.f && u < 0x1p-41f, 0)) u *= 0x1p20f, shift += 20;
  return __umul64hi(__float2ull_rz(u * 0x1p64f), total) >> min(shift, 63);
}

// kWide elements of a row from element i on (0 beyond `end`), kept as loaded; 16-byte
// loads if kVec (then the row is 16-byte aligned and i a multiple of kWide), one element
// otherwise.
template <class T, bool kVec>
struct Wide {
  static constexpr int kWide = kVec ? 16 / (int)sizeof(T) : 1;
  uint32_t w[kVec ? 4 : 1];

  __device__ __forceinline__ void load(const T* row, int i, int end) {
    if constexpr (kVec) {
      if (i + kWide <= end) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + i));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        w[0] = w[1] = w[2] = w[3] = 0u;
#pragma unroll
        for (int k = 0; k < kWide; ++k)
          if (i + k < end) w[k * sizeof(T) / 4] |= bits(row[i + k]) << (8 * (k * sizeof(T) % 4));
      }
    } else {
      w[0] = i < end ? bits(row[i]) : 0u;
    }
  }
  __device__ __forceinline__ float get(int k) const {
    const uint32_t v = w[k * sizeof(T) / 4] >> (8 * (k * sizeof(T) % 4));
    return __uint_as_float(sizeof(T) == 4 ? v : v << 16);
  }
  static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ uint32_t bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace
}  // namespace mla
