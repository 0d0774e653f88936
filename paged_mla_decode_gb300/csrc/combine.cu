// combine.cu -- log-sum-exp merge of partial attention results.
//
// "vLLM x AgentX: Optimizing for Real-World Agentic Serving", section "Kimi
// K3": partial attention outputs over disjoint pieces of a sequence carry
// their log-sum-exp statistics and are merged with online softmax:
//   lse = ln sum_s exp(lse_s),  out = sum_s exp(lse_s - lse) * out_s.
// A piece with lse_s = -inf (empty) contributes nothing; a row whose pieces
// are all empty (or that is flagged bad) gets out = 0 and lse = -inf.
// A piece with a NaN (lse_s = +inf in a decode's partials, NaN in its results)
// makes the row NaN.
#include <algorithm>
#include <atomic>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "merge_pieces.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kCombineThreads = 128;  // 4 output dims per thread

// Merges `np` partials of one (row, head). Partial s sits at
// out_base + s*out_stride (512 floats) and lse_base + s*lse_stride.
// Every thread handles output dims [4*tid, 4*tid+4). s_w holds np floats.
__device__ __forceinline__ void merge_row(const float* __restrict__ out_base, int64_t out_stride,
                                          const float* __restrict__ lse_base, int64_t lse_stride,
                                          int np, bool bad, __nv_bfloat16* __restrict__ out_row,
                                          float* __restrict__ lse_out, float* s_w) {
  __shared__ float s_red[kCombineThreads / 32];
  const int tid = threadIdx.x;
  // (a NaN lse is taken as +inf: a maximum does not pass a NaN on, and the weight
  // exp(inf - inf) is one)
  const auto lse_of = [&](int s) {
    const float l = lse_base[s * lse_stride];
    return isnan(l) ? INFINITY : l;
  };
  float m = -INFINITY;
  if (!bad)
    for (int s = tid; s < np; s += kCombineThreads) m = fmaxf(m, lse_of(s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) s_red[tid >> 5] = m;
  __syncthreads();
  m = s_red[0];
#pragma unroll
  for (int w = 1; w < kCombineThreads / 32; ++w) m = fmaxf(m, s_red[w]);
  __syncthreads();
  const bool empty = bad || !(m > -INFINITY);
  float total = 0.f;
  if (!empty) {
    for (int s = tid; s < np; s += kCombineThreads) {
      const float l = lse_of(s);
      const float w = (l > -INFINITY) ? fast_exp2((l - m) * kLog2e) : 0.f;
      s_w[s] = w;
      total += w;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if ((tid & 31) == 0) s_red[tid >> 5] = total;
  __syncthreads();
  total = 0.f;
#pragma unroll
  for (int w = 0; w < kCombineThreads / 32; ++w) total += s_red[w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!empty) {
    const float inv = 1.0f / total;
    for (int s = 0; s < np; ++s) {
      const float w = s_w[s] * inv;
      if (w == 0.f) continue;  // empty piece: its output is never read
      const float4 v = *reinterpret_cast<const float4*>(out_base + s * out_stride + 4 * tid);
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    }
  }
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
  __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
  uint2 packed;
  packed.x = *reinterpret_cast<uint32_t*>(&lo);
  packed.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(out_row + 4 * tid) = packed;
  if (tid == 0) *lse_out = empty ? -INFINITY : m + logf(total);
}

// ---- merge of a decode's pieces ----
// Units are (row, head, quarter of the 512 dims). With few rows each may have many pieces,
// and every unit is merged by a block (merge_unit: the slices staged by bulk copies).
// Otherwise only the rows of more than kFewPieces pieces are, of which there are at most
// `many_rows` (every CTA's range cuts one row at most), and the other units take a warp
// each: a block would spend its barriers and its staging on a few pieces there. The grid
// then starts with the blocks of the rows of many pieces; each looks for its row in the
// row table and leaves if there is none. A decode call of 256 rows of 8 pages, 64 heads,
// takes 84 us, with a block per unit throughout 178; 48 rows of one page 28 and 42; one
// row of 100k tokens among 31 of one page 101 and 110. For the few rows the first kernel
// stays: it has 32 registers a thread, the second 52 (8 rows of 20k tokens 47 us, 53).
constexpr int kFewPieces = 16;
constexpr int kWarpMergeLoads = 4;  // pieces whose loads are in flight (8: 95 us, 16: 168 on the 256 rows)

struct MergeParams {
  const int32_t* row_base;
  const int32_t* row_np;
  const int32_t* piece_err;
  const float* part_lse;
  const float* part_out;
  int rows, heads;
  int64_t units;
  unsigned many_blocks;  // blocks for rows of many pieces, before the others
  __nv_bfloat16* out;
  float* lse;
  unsigned* status;
  int stage_pieces;
};

// Row number k (from 0) among those of more than kFewPieces pieces; -1 if there are fewer.
// All threads of the block call it; 128 rows a warp at a time.
__device__ __forceinline__ int find_row_of_many(const MergeParams& p, int k) {
  __shared__ int s_count[kMergeWarps];
  __shared__ int s_found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_found = -1;
  for (int r0 = 0; r0 < p.rows; r0 += 128 * kMergeWarps) {
    unsigned many[4];
    int count = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + 128 * warp + 32 * j + lane;
      many[j] = __ballot_sync(0xffffffffu, r < p.rows && __ldcg(p.row_np + min(r, p.rows - 1)) > kFewPieces);
      count += __popc(many[j]);
    }
    if (lane == 0) s_count[warp] = count;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) before += s_count[w];
      all += s_count[w];
    }
    int left = k - before;
    if (left >= 0 && left < count && lane == 0) {
      for (int j = 0; j < 4; ++j) {
        const int n = __popc(many[j]);
        if (left < n) {
          s_found = r0 + 128 * warp + 32 * j + (int)__fns(many[j], 0, left + 1);
          break;
        }
        left -= n;
      }
    }
    __syncthreads();
    if (s_found >= 0 || k < all) break;
    k -= all;
  }
  return s_found;
}

// One unit by one warp: lane l keeps dims 4l .. 4l + 3 of its 128, and the weight of one of
// 32 pieces at a time.
__device__ __forceinline__ void merge_unit_by_warp(const MergeParams& p, int64_t unit, int lane) {
  const int quarter = (int)(unit % kMergeQuarters);
  const int64_t rh = unit / kMergeQuarters;
  const int r = (int)(rh / p.heads), h = (int)(rh - (int64_t)r * p.heads);
  const int np = __ldcg(p.row_np + r), base = __ldcg(p.row_base + r);
  if (np > kFewPieces) return;  // another block's
  float l_own = -INFINITY;
  int bad = 0;
  if (lane < np) {
    l_own = __ldcg(p.part_lse + (int64_t)(base + lane) * p.heads + h);
    bad = __ldcg(p.piece_err + base + lane);
  }
  float m = l_own;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool empty = np <= 0 || __any_sync(0xffffffffu, bad != 0) || !(m > -INFINITY);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (!empty) {
    const float* src =
        p.part_out + ((int64_t)base * p.heads + h) * kDLatent + 128 * quarter + 4 * lane;
    const int64_t step = (int64_t)p.heads * kDLatent;
    const float w_own = l_own > -INFINITY ? fast_exp2((l_own - m) * kLog2e) : 0.f;
    for (int k0 = 0; k0 < np; k0 += kWarpMergeLoads) {
      float4 v[kWarpMergeLoads];
#pragma unroll
      for (int k = 0; k < kWarpMergeLoads; ++k)
        if (k0 + k < np) v[k] = __ldcg(reinterpret_cast<const float4*>(src + (k0 + k) * step));
#pragma unroll
      for (int k = 0; k < kWarpMergeLoads; ++k) {
        if (k0 + k >= np) break;
        const float w = __shfl_sync(0xffffffffu, w_own, k0 + k);
        if (w == 0.f) continue;  // an empty piece: its slice may hold anything
        acc.x += w * v[k].x; acc.y += w * v[k].y; acc.z += w * v[k].z; acc.w += w * v[k].w;
        total += w;
      }
    }
  }
  const float inv = empty ? 0.f : 1.0f / total;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 packed;
  packed.x = *reinterpret_cast<const uint32_t*>(&lo);
  packed.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p.out + rh * kDLatent + 128 * quarter + 4 * lane) = packed;
  if (quarter == 0 && lane == 0) p.lse[rh] = empty ? -INFINITY : m + logf(total);
}

// Unit `unit` by the whole block.
__device__ __forceinline__ void merge_unit_by_block(const MergeParams& p, int64_t unit) {
  extern __shared__ float4 stage[];                 // [stage_pieces][32] float4
  __shared__ __align__(8) uint64_t mbar;
  __shared__ MergeShared sm;
  const uint32_t mb = smem_u32(&mbar);
  if (threadIdx.x == 0) {
    tc::mbar_init(mb, 1);
    tc::fence_mbar_init();
  }
  uint32_t phase = 0;
  const bool ok = merge_unit(
      unit, p.heads, p.row_base, p.row_np, p.piece_err, p.part_lse, p.part_out, p.out, p.lse,
      p.stage_pieces, stage, sm, mb, phase, (int)threadIdx.x, [] { __syncthreads(); },
      [](bool pred) { return __syncthreads_or(pred ? 1 : 0) != 0; });
  if (!ok && threadIdx.x == 0) atomicOr(p.status, MLA_DEVICE_ERR_TIMEOUT);
}

// Both are launched as dependents of the decode kernel: its partials are visible after
// griddep_wait.
__global__ void __launch_bounds__(kMergeThreads) combine_pieces_kernel(const MergeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  merge_unit_by_block(p, blockIdx.x);
}

__global__ void __launch_bounds__(kMergeThreads) combine_rows_kernel(const MergeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x >= p.many_blocks) {
    const int64_t unit =
        (int64_t)(blockIdx.x - p.many_blocks) * kMergeWarps + (threadIdx.x >> 5);
    if (unit < p.units) merge_unit_by_warp(p, unit, threadIdx.x & 31);
    return;
  }
  const unsigned per_row = (unsigned)p.heads * kMergeQuarters;
  const int row = find_row_of_many(p, (int)(blockIdx.x / per_row));
  if (row >= 0) merge_unit_by_block(p, (int64_t)row * per_row + blockIdx.x % per_row);
}

// Standalone merge: part_out [S][rows][512], part_lse [S][rows]; one block per row.
__global__ void __launch_bounds__(kCombineThreads)
combine_dense_kernel(const float* __restrict__ part_out, const float* __restrict__ part_lse,
                     int num_parts, int64_t rows, __nv_bfloat16* __restrict__ out,
                     float* __restrict__ lse) {
  extern __shared__ float s_w[];
  const int64_t r = blockIdx.x;
  merge_row(part_out + r * kDLatent, rows * kDLatent, part_lse + r, rows, num_parts, false,
            out + r * kDLatent, lse + r, s_w);
}

}  // namespace

cudaError_t launch_combine_pieces(const DecodeWorkspace& ws, int rows, int heads, int passes,
                                  int max_pieces_per_row, __nv_bfloat16* out, float* lse,
                                  cudaStream_t stream) {
  static std::atomic<int> configured[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev].load()) {
    for (const auto kernel : {combine_pieces_kernel, combine_rows_kernel}) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMergeStagePieces * (int)kMergeSliceBytes);
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 64) configured[dev].store(1);
  }
  MergeParams p;
  p.row_base = ws.row_base;
  p.row_np = ws.row_np;
  p.piece_err = ws.piece_err;
  p.part_lse = ws.part_lse;
  p.part_out = ws.part_out;
  p.rows = rows;
  p.heads = heads;
  p.units = (int64_t)rows * heads * kMergeQuarters;
  // a row of more than kFewPieces pieces is cut at least kFewPieces times (kFewPieces - 1
  // if its prefix and suffix pieces count together), and the ranges of a pass's CTAs make
  // fewer cuts than there are CTAs (G of them, which is also the most pieces that a row can
  // have; F forks of one prefix are cut by G / F workers each)
  const int64_t many_rows = (int64_t)passes * max_pieces_per_row / (kFewPieces - 1);
  const bool few_rows = rows <= many_rows;
  p.many_blocks = few_rows ? 0u : (unsigned)(many_rows * heads * kMergeQuarters);
  p.out = out;
  p.lse = lse;
  p.status = ws.status;
  p.stage_pieces = merge_stage_pieces(max_pieces_per_row, rows);
  const int64_t blocks =
      few_rows ? p.units : p.many_blocks + (p.units + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = (size_t)p.stage_pieces * kMergeSliceBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_rows ? combine_pieces_kernel : combine_rows_kernel, p);
}

}  // namespace mla

extern "C" mla_status mla_decode_combine(const float* part_out, const float* part_lse,
                                         int num_parts, int64_t num_rows, void* out, float* lse,
                                         mla_stream_t stream) {
  using namespace mla;
  if (num_parts < 0 || num_rows < 0) return MLA_ERR_INVALID_ARG;
  if (num_rows == 0) return MLA_OK;
  if (!out || !lse) return MLA_ERR_INVALID_ARG;
  if (num_parts > 0 && (!part_out || !part_lse)) return MLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(part_out) & 15u) || (reinterpret_cast<uintptr_t>(out) & 15u) ||
      (reinterpret_cast<uintptr_t>(part_lse) & 3u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MLA_ERR_INVALID_ARG;
  if (num_rows > 0x7fffffffLL) return MLA_ERR_UNSUPPORTED;
  const size_t smem = sizeof(float) * (size_t)max(num_parts, 1);
  if (smem > 200 * 1024) return MLA_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (smem > 48 * 1024) {
    if (cudaFuncSetAttribute(combine_dense_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  combine_dense_kernel<<<(unsigned)num_rows, kCombineThreads, smem, s>>>(
      part_out, part_lse, num_parts, num_rows, static_cast<__nv_bfloat16*>(out), lse);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
