// kv_gather.cu -- read cached entries back as bfloat16 rows.
//
// The read side of "Smaller, faster, safer: running Kimi and GLM at scale", section
// "Quantizing the KV cache" (cached values are converted back as they are read), for
// callers that need the entries themselves, such as a prefill chunk that attends over
// the cached context with up-projected keys and values: packed rows of ragged ranges of
// requests, value(code) * kv_scale in float32, rounded once to bfloat16.
//
// 1,152 bytes written and 297 to 1,152 read per row: DRAM bound, if few instructions are
// spent on 16 bytes of output (4-bit: 5.8 TB/s, e4m3: 6.3, bf16: 6.6). A block takes 32
// rows: it looks their pages up once, then
// a thread keeps one 8-element column of eight of the rows, with all its loads in flight
// before the first store, and a warp stores 512 contiguous bytes. A 4-bit value has 8
// magnitudes times 15 powers, so a block forms those products once, as a table whose row
// is looked up by byte permutes: two per 4 elements instead of conversions and products
// per element.
#include "kv_e2m1.cuh"
#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kVecPerRow = kDEntry / 8;               // a thread writes 8 elements (16 bytes)
constexpr int kGatherThreads = 288;                   // 4 rows at a time
constexpr int kRowsAtOnce = kGatherThreads / kVecPerRow;
// Rows of a thread: eight keep enough loads in flight; two, where a call has few rows,
// spread it over more SMs (1,200 rows: 4.3 us against 6.2; 7,000 rows: 6.2 either way).
constexpr int kBatchMany = 8, kBatchFew = 2;
// Blocks per SM (registers): five of the 4-bit and e4m3 kernels (78 and 85 us for 4
// ranges of 60k-100k rows, 93 and 86 without the bound), three of the bf16 kernel, whose
// loads need the registers (109 us; 144 with five).
template <int kDtype>
constexpr int kGatherBlocks = kDtype == MLA_KV_BF16 ? 3 : 5;

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

// A column (8 elements from 8u on) of one entry: its bytes as loaded, then as bf16.
template <int kDtype>
struct Column;

template <>
struct Column<MLA_KV_BF16> {
  static constexpr int64_t kPage = (int64_t)kPageSize * kDEntry * 2;
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* page, int t, int u) {
    v = __ldg(reinterpret_cast<const uint4*>(page) + t * kVecPerRow + u);
  }
  __device__ __forceinline__ uint4 value(float, const uint4*, int) const { return v; }
};

template <>
struct Column<MLA_KV_E4M3> {
  static constexpr int64_t kPage = (int64_t)kPageSize * kDEntry;
  uint2 c;
  __device__ __forceinline__ void load(const uint8_t* page, int t, int u) {
    c = __ldg(reinterpret_cast<const uint2*>(page) + t * kVecPerRow + u);
  }
  __device__ __forceinline__ uint4 value(float scale, const uint4*, int) const {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e4m3x2_to_f16x2((uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      r[i] = bf16x2_of(f.x * scale, f.y * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

template <>
struct Column<MLA_KV_E2M1> {
  static constexpr int64_t kPage = kE2m1PageBytes;
  uint32_t w, e;
  __device__ __forceinline__ void load(const uint8_t* page, int t, int u) {
    const int b = u >> 2;
    w = __ldg(reinterpret_cast<const uint32_t*>(page + e2m1_code_offset(b, t)) + (u & 3));
    e = __ldg(page + e2m1_exp_offset(b, t));
  }
  // table[n]: the low bytes of the 8 magnitudes' bf16 values, then their high bytes
  __device__ __forceinline__ uint4 value(float, const uint4* table, int u) const {
    const uint4 t = table[((u >> 2) & 1) ? e >> 4 : e & 15u];
    const uint32_t mag = w & 0x77777777u, even = w << 4;
    const uint32_t s0 = __byte_perm(even, w, 0x5140) & 0x80808080u;
    const uint32_t s1 = __byte_perm(even, w, 0x7362) & 0x80808080u;
    const uint32_t l0 = __byte_perm(t.x, t.y, mag), l1 = __byte_perm(t.x, t.y, mag >> 16);
    const uint32_t h0 = __byte_perm(t.z, t.w, mag) | s0, h1 = __byte_perm(t.z, t.w, mag >> 16) | s1;
    return make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362),
                      __byte_perm(l1, h1, 0x5140), __byte_perm(l1, h1, 0x7362));
  }
};

// Words j and 2 + j of table row n: the low and the high bytes of the bf16 values of
// magnitudes 4j .. 4j + 3 times 2^(n - 8) times the scale. The power scales the scale
// exactly, so one float32 product rounds as value * kv_scale.
__device__ __forceinline__ void e2m1_table_words(uint32_t* row, int n, int j, float scale) {
  const float s = n == kE2m1NanExp ? __int_as_float(0x7fffffff)
                                   : scale * __int_as_float((127 - 8 + n) << 23);
  const uint32_t a = j ? bf16x2_of(2.f * s, 3.f * s) : bf16x2_of(0.f * s, 0.5f * s);
  const uint32_t b = j ? bf16x2_of(4.f * s, 6.f * s) : bf16x2_of(s, 1.5f * s);
  row[j] = __byte_perm(a, b, 0x6420);
  row[2 + j] = __byte_perm(a, b, 0x7531);
}

template <int kDtype, int kBatch>
__global__ void __launch_bounds__(kGatherThreads, kGatherBlocks<kDtype>)
    kv_gather_kernel(const GatherParams p) {
  constexpr int kTileRows = kRowsAtOnce * kBatch;
  __shared__ int64_t s_page[kTileRows];  // byte offset of the row's page; -1: a row of zeros
  __shared__ int s_token[kTileRows];     // its token; -1: a row that is left as it was
  __shared__ uint4 s_table[kDtype == MLA_KV_E2M1 ? 16 : 1];
  const int tid = threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * kTileRows;
  if constexpr (kDtype == MLA_KV_E2M1) {
    if (tid >= 32 && tid < 64)  // (the rows are looked up by the first warp)
      e2m1_table_words(reinterpret_cast<uint32_t*>(&s_table[(tid - 32) >> 1]), (tid - 32) >> 1,
                       tid & 1, p.kv_scale);
  }
  if (tid < kTileRows) {
    const int64_t r = r0 + tid;
    int64_t page = -1;
    int token = -1;
    const int32_t begin = __ldg(p.cu), end = __ldg(p.cu + p.batch);
    if (r < p.num_tokens && r >= begin && r < end) {
      int lo = 0, hi = p.batch - 1;  // first request whose rows end after r
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid + 1) > r) hi = mid;
        else lo = mid + 1;
      }
      const int64_t pos = (p.starts ? (int64_t)__ldg(p.starts + lo) : 0) + r - __ldg(p.cu + lo);
      token = 0;
      if (pos >= 0 && pos < (int64_t)p.max_pages * kPageSize) {
        const int64_t id = __ldg(p.block_table + (int64_t)lo * p.max_pages + pos / kPageSize);
        if (id >= 0 && id < p.num_pages) {
          page = id * Column<kDtype>::kPage;
          token = (int)(pos % kPageSize);
        }
      }
    }
    s_page[tid] = page;
    s_token[tid] = token;
  }
  __syncthreads();
  const int u = tid % kVecPerRow, first = tid / kVecPerRow;
  Column<kDtype> c[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int64_t page = s_page[first + kRowsAtOnce * k];
    if (page >= 0) c[k].load(p.kv + page, s_token[first + kRowsAtOnce * k], u);
  }
  const bool is_rope = u >= kDLatent / 8;
  uint4* dst = is_rope ? reinterpret_cast<uint4*>(p.rope) + r0 * (kDRope / 8) + (u - kDLatent / 8)
                       : reinterpret_cast<uint4*>(p.latent) + r0 * (kDLatent / 8) + u;
  const int step = is_rope ? kDRope / 8 : kDLatent / 8;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int row = first + kRowsAtOnce * k;
    if (s_token[row] >= 0)
      dst[row * step] = s_page[row] >= 0 ? c[k].value(p.kv_scale, s_table, u) : make_uint4(0, 0, 0, 0);
  }
}

template <int kDtype>
void launch_gather(const GatherParams& p, cudaStream_t s) {
  const auto blocks = [&](int batch) {
    return (unsigned)((p.num_tokens + kRowsAtOnce * batch - 1) / (kRowsAtOnce * batch));
  };
  if (blocks(kBatchMany) < (unsigned)device_sm_count())
    kv_gather_kernel<kDtype, kBatchFew><<<blocks(kBatchFew), kGatherThreads, 0, s>>>(p);
  else
    kv_gather_kernel<kDtype, kBatchMany><<<blocks(kBatchMany), kGatherThreads, 0, s>>>(p);
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
  if (num_tokens > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
  const GatherParams p{static_cast<const uint8_t*>(kv_pages), num_pages, kv_scale, block_table,
                       max_pages, starts, cu_tokens, batch, num_tokens,
                       static_cast<__nv_bfloat16*>(latent), static_cast<__nv_bfloat16*>(rope)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (kv_dtype == MLA_KV_E2M1) launch_gather<MLA_KV_E2M1>(p, s);
  else if (kv_dtype == MLA_KV_E4M3) launch_gather<MLA_KV_E4M3>(p, s);
  else launch_gather<MLA_KV_BF16>(p, s);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
