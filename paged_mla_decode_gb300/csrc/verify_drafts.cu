// verify_drafts.cu -- accept or reject drafted tokens and sample the next one.
//
// "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
// custom speculative decoding ...": drafted tokens are verified in parallel without
// changing the target model's distribution. Draft j (token x_j, drawn from q_j) is kept
// with probability min(1, p_j(x_j) / q_j(x_j)); at the first rejection the next token is
// drawn from max(p_j - q_j, 0), normalised; if all are kept, from p of the position after
// the last one.
//
// Arithmetic. A probability becomes a 64-bit integer in units of 2^-60 (exact for a
// float32 of 2^-37 and above, truncated below), so that sums are exact, do not depend on
// the order of addition, and the sampled index is the smallest i with
// sum_{k <= i} w_k > u * sum w, decided in integers. The acceptance test compares
// u * q < p in double, where the product is exact.
//
// One row of p (and one of q after a rejection) is read: DRAM bound for many requests,
// latency bound for few. So a request is worked by a cluster of up to eight blocks, each
// summing a run of the vocabulary; the blocks exchange their sums through distributed
// shared memory, and the one whose run holds the border scans the 1/16 of it (a warp's
// run) that does, with all its threads at once.
#include <algorithm>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 2;  // tiles of a warp in flight: 32 KB of p and q per block, two blocks an SM

struct VerifyParams {
  const void* target;
  int64_t target_stride;  // elements between rows
  const void* draft;      // may be null: the drafter puts all its weight on the draft
  int64_t draft_stride;
  const int32_t* tokens;
  const float* uniforms;
  const int32_t* num_drafts;  // may be null: max_drafts each
  const int32_t* seq_lens;    // may be null
  int batch, max_drafts, vocab;
  int32_t* out_tokens;
  int32_t* accepted;
  int32_t* seq_lens_out;      // may be null
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// A probability within [0, 1] (NaN and negative values: 0).
__device__ __forceinline__ float weight(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
__device__ __forceinline__ uint64_t fixed60(float x) { return __float2ull_rz(weight(x) * 0x1p60f); }
__device__ __forceinline__ float unit(float u) { return u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f; }

// The distribution that the next token is drawn from: p, or what a rejection leaves of it.
template <class T>
struct Rest {
  const T* p;
  const T* q;  // null: none, or all of `skip`'s weight
  int skip;    // token that lost all its weight (-1: none)

  __device__ __forceinline__ uint64_t of(float pi, float qi, int i) const {
    const uint64_t a = fixed60(pi);
    if (q == nullptr) return i == skip ? 0 : a;
    const uint64_t b = fixed60(qi);
    return a > b ? a - b : 0;
  }
};

// kWide elements of a row from element i on (0 beyond `end`); 16-byte loads if kVec (then
// the row is 16-byte aligned and i a multiple of kWide), one element otherwise.
template <class T, bool kVec>
struct Wide {
  static constexpr int kWide = kVec ? 16 / (int)sizeof(T) : 1;
  static __device__ __forceinline__ void load(const T* row, int i, int end, float (&x)[kWide]) {
    if (kVec && i + kWide <= end) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + i));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < kWide; ++k) {
        if constexpr (sizeof(T) == 4) x[k] = __uint_as_float(w[k % 4]);
        else x[k] = __uint_as_float((k & 1) ? w[(k / 2) % 4] & 0xffff0000u : w[(k / 2) % 4] << 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kWide; ++k) x[k] = i + k < end ? to_float(row[i + k]) : 0.f;
    }
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kVerifyThreads, 2)
    verify_kernel(const VerifyParams p, const int run) {
  using W = Wide<T, kVec>;
  constexpr int kTile = 32 * W::kWide;  // elements a warp takes at a time
  __shared__ uint64_t s_warp[kVerifyWarps];  // sums of the warps' runs
  __shared__ uint64_t s_block[2];            // of the block's, by pass; read by the cluster
  __shared__ uint64_t s_scan[kVerifyWarps];
  __shared__ int s_row, s_token;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ranks, K = p.max_drafts, V = p.vocab;
  const int drafts = p.num_drafts ? p.num_drafts[b] : K;
  const int L = p.seq_lens ? p.seq_lens[b] : 0;
  int32_t* out = p.out_tokens + (int64_t)b * (K + 1);
  if (drafts < 0 || drafts > K || L < 0) {  // left out: nothing of it changes the length
    if (rank == 0) {
      for (int i = tid; i <= K; i += kVerifyThreads) out[i] = -1;
      if (tid == 0) {
        p.accepted[b] = -1;
        if (p.seq_lens_out) p.seq_lens_out[b] = L;
      }
    }
    return;
  }
  const T* target = static_cast<const T*>(p.target) + (int64_t)b * (K + 1) * p.target_stride;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + (int64_t)b * K * p.draft_stride : nullptr;
  const float* u = p.uniforms + (int64_t)b * (K + 1);
  const int32_t* tokens = p.tokens + (int64_t)b * K;
  if (warp == 0) {
    bool ok = false;
    if (lane < drafts) {
      const int x = tokens[lane];
      if (x >= 0 && x < V) {
        const float px = weight(to_float(target[lane * p.target_stride + x]));
        const float qx = draft ? weight(to_float(draft[lane * p.draft_stride + x])) : 1.f;
        ok = (double)unit(u[lane]) * (double)qx < (double)px;
      }
    }
    const int kept = __ffs(~__ballot_sync(0xffffffffu, ok)) - 1;  // K <= 31: some lane is false
    if (lane == 0) {
      s_row = kept;
      s_token = -1;
    }
  }
  __syncthreads();
  const int a = s_row;
  const bool rejected = a < drafts;
  Rest<T> rest{target + a * p.target_stride,
               rejected && draft ? draft + a * p.draft_stride : nullptr,
               rejected && !draft ? tokens[a] : -1};
  // this warp's run of the vocabulary
  const int lo = (int)min((int64_t)(rank * kVerifyWarps + warp) * run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + run, (int64_t)V);
  uint64_t total = 0, before = 0;  // of all blocks; of those before this one
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;
    for (int i0 = lo; i0 < hi; i0 += kUnroll * kTile) {
      float pi[kUnroll][W::kWide], qi[kUnroll][W::kWide];
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        const int i = i0 + t * kTile + lane * W::kWide;
        W::load(rest.p, i, hi, pi[t]);
        if (rest.q != nullptr) W::load(rest.q, i, hi, qi[t]);
      }
#pragma unroll
      for (int t = 0; t < kUnroll; ++t)
#pragma unroll
        for (int k = 0; k < W::kWide; ++k)
          sum += rest.of(pi[t][k], qi[t][k], i0 + t * kTile + lane * W::kWide + k);
    }
    sum = warp_sum(sum);
    __syncthreads();  // (the last pass's sums are no longer read)
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const uint64_t all = warp_sum(lane < kVerifyWarps ? s_warp[lane] : 0);
      if (lane == 0) s_block[pass] = all;
    }
    cluster.sync();
    total = before = 0;
    for (int r = 0; r < ranks; ++r) {
      const uint64_t v = *cluster.map_shared_rank(&s_block[pass], r);
      total += v;
      if (r < rank) before += v;
    }
    if (total > 0 || !rejected) break;
    rest.q = nullptr;  // a rejection that leaves nothing: the target's own distribution
    rest.skip = -1;
  }
  // no block leaves while another may still read its sums, and every block has read the
  // length that block 0 may overwrite
  cluster.sync();
  if (rank == 0) {
    for (int i = tid; i <= K; i += kVerifyThreads)
      if (i != a) out[i] = i < a ? tokens[i] : -1;
    if (tid == 0) {
      if (total == 0) out[a] = -1;
      p.accepted[b] = a;
      if (p.seq_lens_out) p.seq_lens_out[b] = L - (drafts - a);
    }
  }
  // the border: the first token whose running sum exceeds u * total, in integers
  const uint64_t at = __umul64hi(__float2ull_rz(unit(u[K]) * 0x1p64f), total);
  int w = 0;
  while (w < kVerifyWarps && before + s_warp[w] <= at) before += s_warp[w++];
  if (total == 0 || at < before || w == kVerifyWarps) return;  // in another block's run
  const int run_lo = (int)min((int64_t)(rank * kVerifyWarps + w) * run, (int64_t)V);
  const int run_hi = (int)min((int64_t)run_lo + run, (int64_t)V);
  for (int i0 = run_lo; i0 < run_hi; i0 += kVerifyThreads * W::kWide) {
    const int i = i0 + tid * W::kWide;
    float pi[W::kWide], qi[W::kWide];
    W::load(rest.p, i, run_hi, pi);
    if (rest.q != nullptr) W::load(rest.q, i, run_hi, qi);
    uint64_t mine = 0;
#pragma unroll
    for (int k = 0; k < W::kWide; ++k) mine += rest.of(pi[k], qi[k], i + k);
    uint64_t c = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += v;
    }
    if (lane == 31) s_scan[warp] = c;
    __syncthreads();
    uint64_t upto = before;  // sum before this thread's elements
    for (int k = 0; k < warp; ++k) upto += s_scan[k];
    upto += c - mine;
    if (upto <= at && at < upto + mine) {  // one thread at most
      int k = 0;
#pragma unroll
      for (int j = 0; j < W::kWide; ++j) {
        const uint64_t v = rest.of(pi[j], qi[j], i + j);
        if (upto + v <= at) {
          upto += v;
          k = j + 1;
        } else {
          upto = ~0ull;  // past the border: every later test fails
          break;
        }
      }
      s_token = i + k;
    }
    uint64_t all = 0;
    for (int k = 0; k < kVerifyWarps; ++k) all += s_scan[k];
    before += all;
    __syncthreads();
    if (at < before) break;
  }
  if (tid == 0) out[a] = s_token;
}

// Blocks per request: as many as keep 2,048 tokens each, so that few requests still
// spread over many SMs. On 131,072 tokens and one request VERIFY_NUMBERS
int cluster_blocks(int vocab) {
  int c = 1;
  while (c < kMaxCluster && vocab >= 2 * c * 2048) c *= 2;
  return c;
}

template <class T, bool kVec>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  const int ranks = cluster_blocks(p.vocab);
  constexpr int kTile = 32 * Wide<T, kVec>::kWide;
  const int warps = ranks * kVerifyWarps;
  const int run = (int)(((int64_t)p.vocab + (int64_t)warps * kTile - 1) / ((int64_t)warps * kTile)) * kTile;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * ranks));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, kVec>, p, run);
}

template <class T>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  // 16-byte loads where every row starts on a 16-byte boundary
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.target) | reinterpret_cast<uintptr_t>(p.draft);
  const int64_t strides = (p.target_stride | (p.draft ? p.draft_stride : 0)) * (int64_t)sizeof(T);
  return ((at | (uintptr_t)strides) & 15u) == 0 ? launch_verify<T, true>(p, stream)
                                                : launch_verify<T, false>(p, stream);
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_verify_drafts(const void* target_probs, int64_t target_stride,
                                        const void* draft_probs, int64_t draft_stride,
                                        int prob_dtype, const int32_t* draft_tokens,
                                        const float* uniforms, const int32_t* num_drafts,
                                        const int32_t* seq_lens, int batch, int max_drafts,
                                        int vocab, int32_t* out_tokens, int32_t* num_accepted,
                                        int32_t* seq_lens_out, mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || max_drafts < 0 || max_drafts > MLA_MAX_DRAFTS || vocab < 1)
    return MLA_ERR_INVALID_ARG;
  if (prob_dtype != MLA_PROB_F32 && prob_dtype != MLA_PROB_BF16) return MLA_ERR_INVALID_ARG;
  if (batch > 0x7fffffff / kMaxCluster || vocab > 1 << 30) return MLA_ERR_UNSUPPORTED;
  if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return MLA_ERR_INVALID_ARG;
  if (seq_lens_out && !seq_lens) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!target_probs || !uniforms || !out_tokens || !num_accepted ||
      (max_drafts > 0 && !draft_tokens))
    return MLA_ERR_INVALID_ARG;
  const uintptr_t pa = prob_dtype == MLA_PROB_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs)) & pa)
    return MLA_ERR_INVALID_ARG;
  const void* ptrs[7] = {draft_tokens, uniforms,     num_drafts,  seq_lens,
                         out_tokens,   num_accepted, seq_lens_out};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MLA_ERR_INVALID_ARG;
  const VerifyParams p{target_probs, target_stride, max_drafts > 0 ? draft_probs : nullptr,
                       draft_stride, draft_tokens,  uniforms,
                       num_drafts,   seq_lens,      batch,
                       max_drafts,   vocab,         out_tokens,
                       num_accepted, seq_lens_out};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = prob_dtype == MLA_PROB_F32 ? launch_verify<float>(p, s)
                                                   : launch_verify<__nv_bfloat16>(p, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
