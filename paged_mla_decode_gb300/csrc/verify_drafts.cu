// verify_drafts.cu -- accept or reject drafted tokens and sample the next one.
//
// "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
// custom speculative decoding ...": drafted tokens are verified in parallel without
// changing the target model's distribution. Draft j (token x_j, drawn from q_j) is kept
// with probability min(1, p_j(x_j) / q_j(x_j)); at the first rejection the next token is
// drawn from max(p_j - q_j, 0), normalised; if all are kept, from p of the position after
// the last one.
//
// Arithmetic. A probability becomes an integer in units of 2^-60 (exact for a float32 of
// 2^-37 and above, rounded below), so that sums are exact, do not depend on the order of
// addition, and the sampled index is the smallest i with sum_{k <= i} w_k > u * sum w,
// decided in integers. The acceptance test compares u * q < p in double, where the
// product is exact.
//
// One row of p (and one of q after a rejection) is read: bound by DRAM and by the 20
// instructions that a pair of probabilities takes for many requests (4.7 TB/s with 512),
// by latency for few (10 us: the drafts' probabilities, the run, the cluster's exchange,
// the final scan, one after the other). So a request is worked by a cluster of up to eight blocks, each
// summing a run of the vocabulary; the blocks exchange their sums through distributed
// shared memory, and the one whose run holds the border scans the warp's run that does (1/16
// or 1/8 of its own, by the shape of block), with all its threads at once.
#include <algorithm>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
// Two shapes of block. With few requests a block has an SM to itself and every load of a
// run should be in flight at once; with many, four smaller blocks an SM cover each
// other's waits (the drafts' probabilities, the cluster's barriers, the final scan).
struct Few {
  static constexpr int kThreads = 512, kBlocksPerSm = 1, kLoads = 8;  // in flight per row and thread
};
struct Many {
  static constexpr int kThreads = 256, kBlocksPerSm = 4, kLoads = 4;
};

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

// The distribution that the next token is drawn from: p, or what a rejection leaves of it.
template <class T>
struct Rest {
  const T* p;
  const T* q;  // null: none, or all of `skip`'s weight
  int skip;    // token that lost all its weight (-1: none)
};
// Adds a token's weight: max(x - y, 0) with a q row (kPair), x without.
template <bool kPair>
__device__ __forceinline__ void add_weight(Slices& to, float x, float y) {
  const Slices a = slices(weight(x));
  if constexpr (kPair) {
    const Slices b = slices(weight(y));
    if (weight(x) > weight(y)) {
#pragma unroll
      for (int j = 0; j < 3; ++j) to.s[j] += a.s[j] - b.s[j];
    }
  } else {
    const Slices zero = slices(0.f);
#pragma unroll
    for (int j = 0; j < 3; ++j) to.s[j] += a.s[j] - zero.s[j];
  }
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

// Sum of a lane's share of elements lo .. hi - 1 of the row (kUnroll tiles in flight).
template <class T, bool kVec, int kUnroll, bool kPair>
__device__ __forceinline__ uint64_t run_sum(const Rest<T>& rest, int lo, int hi, int lane) {
  using W = Wide<T, kVec>;
  constexpr int kTile = 32 * W::kWide;  // elements a warp takes at a time
  static_assert(kUnroll * W::kWide <= 64, "20-bit slices of 64 elements stay within 32 bits");
  uint64_t sum = 0;
  for (int i0 = lo; i0 < hi; i0 += kUnroll * kTile) {
    W pi[kUnroll], qi[kPair ? kUnroll : 1];
#pragma unroll
    for (int t = 0; t < kUnroll; ++t) {
      const int i = i0 + t * kTile + lane * W::kWide;
      pi[t].load(rest.p, i, hi);
      if constexpr (kPair) qi[t].load(rest.q, i, hi);
    }
    Slices part{{0, 0, 0}};
#pragma unroll
    for (int t = 0; t < kUnroll; ++t)
#pragma unroll
      for (int k = 0; k < W::kWide; ++k)
        add_weight<kPair>(part, pi[t].get(k), kPair ? qi[kPair ? t : 0].get(k) : 0.f);
    sum += joined(part);
  }
  return sum;
}

template <class T>
__device__ __forceinline__ uint64_t weight_of(const T* row, int i) {
  Slices one{{0, 0, 0}};
  add_weight<false>(one, to_float(row[i]), 0.f);
  return joined(one);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <class T, bool kVec, class Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kBlocksPerSm)
    verify_kernel(const VerifyParams p, const int run) {
  using W = Wide<T, kVec>;
  constexpr int kVerifyThreads = Shape::kThreads, kVerifyWarps = kVerifyThreads / 32;
  // tiles of a warp in flight (bf16: twice the elements a load, half the loads)
  constexpr int kUnroll = kVec ? Shape::kLoads * (int)sizeof(T) / 4 : 8;
  __shared__ uint64_t s_warp[kVerifyWarps];  // sums of the warps' runs
  __shared__ uint64_t s_block[2];            // of the block's, by pass; read by the cluster
  __shared__ uint64_t s_scan[kVerifyWarps];
  __shared__ int s_row, s_token;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ranks, K = p.max_drafts, V = p.vocab;
  // everything that hangs on no other load first: one draft a lane
  const int drafts = p.num_drafts ? p.num_drafts[b] : K;
  const int L = p.seq_lens ? p.seq_lens[b] : 0;
  const T* target = static_cast<const T*>(p.target) + (int64_t)b * (K + 1) * p.target_stride;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + (int64_t)b * K * p.draft_stride : nullptr;
  const float* u = p.uniforms + (int64_t)b * (K + 1);
  const int32_t* tokens = p.tokens + (int64_t)b * K;
  const float u_sample = u[K];
  if (warp == 0) {
    bool ok = false;
    if (lane < K) {
      const int x = tokens[lane];
      const float v = unit(u[lane]);
      if (x >= 0 && x < V) {
        const float px = weight(to_float(target[lane * p.target_stride + x]));
        const float qx = draft ? weight(to_float(draft[lane * p.draft_stride + x])) : 1.f;
        ok = lane < drafts && (double)v * (double)qx < (double)px;
      }
    }
    const int kept = __ffs(~__ballot_sync(0xffffffffu, ok)) - 1;  // K <= 31: some lane is false
    if (lane == 0) {
      s_row = kept;
      s_token = -1;
    }
  }
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
  __syncthreads();
  const int a = s_row;
  // -1 unless some block finds the border; that block's store comes after the barrier below
  if (rank == 0 && tid == 0) out[a] = -1;
  const bool rejected = a < drafts;
  Rest<T> rest{target + a * p.target_stride,
               rejected && draft ? draft + a * p.draft_stride : nullptr,
               rejected && !draft ? tokens[a] : -1};
  // this warp's run of the vocabulary
  const int lo = (int)min((int64_t)(rank * kVerifyWarps + warp) * run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + run, (int64_t)V);
  uint64_t total = 0, before = 0;  // of all blocks; of those before this one
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = rest.q != nullptr ? run_sum<T, kVec, kUnroll, true>(rest, lo, hi, lane)
                                     : run_sum<T, kVec, kUnroll, false>(rest, lo, hi, lane);
    if (rest.skip >= lo && rest.skip < hi && lane == 0) sum -= weight_of(rest.p, rest.skip);
    sum = warp_sum(sum);
    __syncthreads();  // (the last pass's sums are no longer read)
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const uint64_t all = warp_sum(lane < kVerifyWarps ? s_warp[lane] : 0);
      if (lane == 0) s_block[pass] = all;
    }
    cluster.sync();
    // lane r reads block r's sum
    const uint64_t v = lane < ranks ? *cluster.map_shared_rank(&s_block[pass], lane) : 0;
    total = warp_sum(v);
    before = warp_sum(lane < rank ? v : 0);
    if (total > 0 || !rejected) break;
    rest.q = nullptr;  // a rejection that leaves nothing: the target's own distribution
    rest.skip = -1;
  }
  // no block leaves while another may still read its sums: arrive here, wait at the end
  cluster.barrier_arrive();
  if (rank == 0) {  // (every block has read the length that may be overwritten here)
    for (int i = tid; i <= K; i += kVerifyThreads)
      if (i != a) out[i] = i < a ? tokens[i] : -1;
    if (tid == 0) {
      p.accepted[b] = a;
      if (p.seq_lens_out) p.seq_lens_out[b] = L - (drafts - a);
    }
  }
  // the border: the first token whose running sum exceeds u * total, in integers
  const uint64_t at = share(unit(u_sample), total);
  int w = 0;
  while (w < kVerifyWarps && before + s_warp[w] <= at) before += s_warp[w++];
  if (total == 0 || at < before || w == kVerifyWarps) {  // in another block's run
    cluster.barrier_wait();
    return;
  }
  const int run_lo = (int)min((int64_t)(rank * kVerifyWarps + w) * run, (int64_t)V);
  const int run_hi = (int)min((int64_t)run_lo + run, (int64_t)V);
  for (int i0 = run_lo; i0 < run_hi; i0 += kVerifyThreads * W::kWide) {
    const int i = i0 + tid * W::kWide;
    W pi, qi;
    pi.load(rest.p, i, run_hi);
    if (rest.q != nullptr) qi.load(rest.q, i, run_hi);
    uint64_t mine = 0, each[W::kWide];
#pragma unroll
    for (int k = 0; k < W::kWide; ++k) {
      Slices one{{0, 0, 0}};
      if (rest.q != nullptr) add_weight<true>(one, pi.get(k), qi.get(k));
      else if (i + k != rest.skip) add_weight<false>(one, pi.get(k), 0.f);
      each[k] = joined(one);
      mine += each[k];
    }
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
        if (upto + each[j] <= at) {
          upto += each[j];
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
  cluster.barrier_wait();
}

// Blocks per request: as many as keep 2,048 tokens each, so that few requests still
// spread over many SMs. Fewer blocks with many requests (one wave of them) were no faster:
// 128 requests of 163,840 tokens 36.3 us with four, 35.7 with eight; 512 120 and 104.
int cluster_blocks(int vocab) {
  int c = 1;
  while (c < kMaxCluster && vocab >= 2 * c * 2048) c *= 2;
  return c;
}

template <class T, bool kVec, class Shape>
cudaError_t launch_verify(const VerifyParams& p, int ranks, cudaStream_t stream) {
  constexpr int kTile = 32 * Wide<T, kVec>::kWide;
  const int64_t share = (int64_t)ranks * (Shape::kThreads / 32) * kTile;
  const int run = (int)((p.vocab + share - 1) / share) * kTile;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * ranks));
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, kVec, Shape>, p, run);
}

template <class T>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  const int sms = device_sm_count(), ranks = cluster_blocks(p.vocab);
  // (19 requests of 131,072 tokens, 152 blocks: 16.6 us, 14.5 with the other shape)
  const bool few = 2 * (int64_t)p.batch * ranks <= sms;
  // 16-byte loads where every row starts on a 16-byte boundary
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.target) | reinterpret_cast<uintptr_t>(p.draft);
  const int64_t strides = (p.target_stride | (p.draft ? p.draft_stride : 0)) * (int64_t)sizeof(T);
  if (((at | (uintptr_t)strides) & 15u) == 0)
    return few ? launch_verify<T, true, Few>(p, ranks, stream)
               : launch_verify<T, true, Many>(p, ranks, stream);
  return few ? launch_verify<T, false, Few>(p, ranks, stream)
             : launch_verify<T, false, Many>(p, ranks, stream);
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
