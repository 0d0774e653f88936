// kv_gather.cu -- read cached entries back as bfloat16 rows.
//
// The read side of "Smaller, faster, safer: running Kimi and GLM at scale", section
// "Quantizing the KV cache" (cached values are converted back as they are read), for
// callers that need the entries themselves, such as a prefill chunk that attends over
// the cached context with up-projected keys and values: packed rows of ragged ranges of
// requests, value(code) * kv_scale in float32, rounded once to bfloat16.
#include "kv_e2m1.cuh"
#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kVecPerRow = kDEntry / 8;  // a thread writes 8 elements (16 bytes)
constexpr int kGatherThreads = 288;      // 4 rows per block

struct GatherParams {
  const uint8_t* kv;
  int64_t num_pages;
  float kv_scale;
  const int32_t* block_table;
  int max_pages;
  const int32_t* starts;  // may be null: every range starts at token 0
  const int32_t* cu;
  int batch;
  int64_t num_tokens;
  __nv_bfloat16* latent;
  __nv_bfloat16* rope;
};

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 f16x2_value(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two e2m1 codes (the low byte of `pair`) -> f16 pair, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t pair) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.u8.u32 b, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}\n" : "=r"(r) : "r"(pair));
  return r;
}

// Elements 8u .. 8u + 7 of the entry at (page, token t) as bf16. The powers of two of a
// 4-bit block scale kv_scale exactly, so one float32 product rounds as value * kv_scale.
template <int kDtype>
__device__ __forceinline__ uint4 load_chunk(const GatherParams& p, int64_t page, int t, int u) {
  if constexpr (kDtype == MLA_KV_BF16) {
    return __ldg(reinterpret_cast<const uint4*>(p.kv) + (page * kPageSize + t) * kVecPerRow + u);
  } else if constexpr (kDtype == MLA_KV_E4M3) {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.kv) + (page * kPageSize + t) * kVecPerRow + u);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? c.x : c.y;
      const float2 v = f16x2_value(e4m3x2_to_f16x2((uint16_t)(w >> (16 * (i & 1)))));
      r[i] = bf16x2_of(v.x * p.kv_scale, v.y * p.kv_scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  } else {
    const int b = u >> 2;
    const uint8_t* base = p.kv + page * kE2m1PageBytes;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(base + e2m1_code_offset(b, t)) + (u & 3));
    const uint32_t e = __ldg(base + e2m1_exp_offset(b, t));
    const uint32_t n = (b & 1) ? e >> 4 : e & 15u;
    const float s = n == kE2m1NanExp ? __int_as_float(0x7fffffff)
                                     : p.kv_scale * __int_as_float((127 - 8 + (int)n) << 23);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = f16x2_value(e2m1x2_to_f16x2((w >> (8 * i)) & 0xffu));
      r[i] = bf16x2_of(v.x * s, v.y * s);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const GatherParams p) {
  const int64_t gid = (int64_t)blockIdx.x * kGatherThreads + threadIdx.x;
  const int64_t r = gid / kVecPerRow;
  const int u = (int)(gid - r * kVecPerRow);
  if (r >= p.num_tokens || r < p.cu[0] || r >= p.cu[p.batch]) return;
  int lo = 0, hi = p.batch - 1;  // first request whose rows end after r
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid + 1) > r) hi = mid;
    else lo = mid + 1;
  }
  const int64_t pos = (p.starts ? (int64_t)__ldg(p.starts + lo) : 0) + r - __ldg(p.cu + lo);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (pos >= 0 && pos < (int64_t)p.max_pages * kPageSize) {
    const int64_t page = __ldg(p.block_table + (int64_t)lo * p.max_pages + pos / kPageSize);
    if (page >= 0 && page < p.num_pages) v = load_chunk<kDtype>(p, page, (int)(pos % kPageSize), u);
  }
  uint4* dst = u < kDLatent / 8
                   ? reinterpret_cast<uint4*>(p.latent) + r * (kDLatent / 8) + u
                   : reinterpret_cast<uint4*>(p.rope) + r * (kDRope / 8) + (u - kDLatent / 8);
  *dst = v;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace mla

extern "C" mla_status mla_kv_gather(const void* kv_pages, int64_t num_pages, int page_size,
                                    int kv_dtype, float kv_scale, const int32_t* block_table,
                                    int max_pages, const int32_t* starts,
                                    const int32_t* cu_tokens, int batch, int64_t num_tokens,
                                    void* latent, void* rope, mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || num_pages < 0 || max_pages < 1 || num_tokens < 0) return MLA_ERR_INVALID_ARG;
  if (page_size != kPageSize) return MLA_ERR_UNSUPPORTED;
  if (kv_dtype != MLA_KV_E4M3 && kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_E2M1)
    return MLA_ERR_INVALID_ARG;
  if (!(kv_scale > 0.0f) || !isfinite(kv_scale)) return MLA_ERR_INVALID_ARG;
  if (kv_dtype == MLA_KV_BF16 && kv_scale != 1.0f) return MLA_ERR_INVALID_ARG;
  if (kv_dtype == MLA_KV_E2M1 && !e2m1_scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return MLA_OK;
  if (!kv_pages || !block_table || !cu_tokens || !latent || !rope) return MLA_ERR_INVALID_ARG;
  if (misaligned(kv_pages, 16) || misaligned(latent, 16) || misaligned(rope, 16) ||
      misaligned(block_table, 4) || misaligned(cu_tokens, 4) || misaligned(starts, 4))
    return MLA_ERR_INVALID_ARG;
  const int64_t grid = (num_tokens * kVecPerRow + kGatherThreads - 1) / kGatherThreads;
  if (num_tokens > 0x7fffffffLL || grid > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
  const GatherParams p{static_cast<const uint8_t*>(kv_pages), num_pages, kv_scale, block_table,
                       max_pages, starts, cu_tokens, batch, num_tokens,
                       static_cast<__nv_bfloat16*>(latent), static_cast<__nv_bfloat16*>(rope)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (kv_dtype == MLA_KV_E2M1)
    kv_gather_kernel<MLA_KV_E2M1><<<(unsigned)grid, kGatherThreads, 0, s>>>(p);
  else if (kv_dtype == MLA_KV_E4M3)
    kv_gather_kernel<MLA_KV_E4M3><<<(unsigned)grid, kGatherThreads, 0, s>>>(p);
  else
    kv_gather_kernel<MLA_KV_BF16><<<(unsigned)grid, kGatherThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
