// logits_probs.cu -- logits to probabilities: penalties, biases, a grammar's mask, softmax.
//
// The step before drafts are verified ("How to serve trillions of tokens for
// trillion-parameter coding agents", section "Use custom speculative decoding ...":
// drafted tokens are verified in parallel without changing the target model's
// distribution, which is the one that a request's sampling settings make of the logits).
// For a row x, token v with count n(v) so far:
//   seen(v) = n(v) > 0 or v in the prompt:  x <- x > 0 ? x / repetition : x * repetition
//   n(v) > 0:                               x <- x - frequency n(v) - presence
//   x <- x + the biases of v;  x <- -inf where the grammar does not allow v
//   p = exp((x - max x) / temperature) / sum
// A drafted token's row also counts the drafts on its own path (the node mask's bits).
//
// A row is read once and written once, so DRAM bounds many rows. A cluster of up to eight
// blocks works a row in two passes over its logits: the first keeps a running maximum and
// sum in every thread, which the blocks exchange through distributed shared memory; the second, which
// finds the logits in L2, writes exp(x - max) / sum. Nothing is staged, so many blocks share an SM
// and one's loads cover another's barriers. Tokens that a list names (biases, drafts) are left
// out of the first pass, by a bit each, and worked out by a thread an entry, which adds up all of
// its token's entries in order: two entries of a token come to the same value.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
// Two shapes of block. With few rows a block has an SM to itself and most of its loads should
// be in flight at once; with many, several smaller blocks an SM cover each other's waits.
struct Few {
  static constexpr int kThreads = 1024, kBlocksPerSm = 1, kUnroll = 2;
};
struct Many {
  static constexpr int kThreads = 256, kBlocksPerSm = 5, kUnroll = 1;
};


struct ProbsParams {
  const void* logits;
  int64_t logit_stride;  // elements between rows
  void* probs;
  int64_t prob_stride;
  int batch, rows, vocab;
  const float* temperature;  // [batch]; this and all below may be null
  const int32_t* num_rows;
  const int32_t* node_tokens;
  const uint64_t* tree_mask;
  const int32_t* counts;
  const uint32_t* prompt;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_tokens;
  const float* biases;
  int num_biases;
  const uint32_t* allowed;
  int words;  // of a row of `prompt` and `allowed`
  int run;    // tokens of a block
  int penalties;
};

// What changes a row's logits, the same for all of its tokens.
struct RowSettings {
  float repetition, inverse, frequency, presence;
  const int32_t* counts;     // of the request; may be null
  const uint32_t* prompt;    // may be null
  const uint32_t* allowed;   // of the row; may be null
};

// (x / repetition is x times its rounded inverse: one more rounding of 2^-24, no division
// for each token)
__device__ __forceinline__ float penalised(float x, int count, bool in_prompt, const RowSettings& s) {
  const float f = x > 0.f ? s.inverse : s.repetition;
  if (count > 0 || in_prompt) x *= f;
  if (count > 0) x = x - fmaf(s.frequency, (float)count, s.presence);
  return x;
}
__device__ __forceinline__ bool bit_of(const uint32_t* words, int v) {
  return (__ldg(words + (v >> 5)) >> (v & 31)) & 1u;
}

template <class T>
struct Eight;  // eight neighbouring elements of a row
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Running maximum and sum of exp((x - max) / t); greedy: the lowest token with the maximum.
struct Stats {
  float max, sum;
  int first;
};

// exp((x - m) / t) for x <= m < inf, m > -inf, with k = 2 log2(e) / t (of half the
// difference, which does not overflow)
__device__ __forceinline__ float weight_of(float x, float m, float k) {
  return fast_exp2(fmaf(0.5f, x, -0.5f * m) * k);
}
// the same for any m: beside an infinite maximum only its equals have a weight
__device__ __forceinline__ float weight_of_any(float x, float m, float k) {
  if (x == m) return m > -INFINITY ? 1.f : 0.f;
  return m == INFINITY || x == -INFINITY ? 0.f : weight_of(x, m, k);
}

template <int kCount>
__device__ __forceinline__ void add_tokens(Stats& s, const float (&x)[kCount], int token, bool greedy, float k) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < kCount; ++e) top = fmaxf(top, x[e]);
  if (top > s.max) {
    s.sum = s.max > -INFINITY ? s.sum * weight_of_any(s.max, top, k) : 0.f;
    s.max = top;
    if (greedy) {
#pragma unroll
      for (int e = kCount - 1; e >= 0; --e)
        if (x[e] == top) s.first = token + e;
    }
  }
  if (greedy || s.max == -INFINITY) return;
  if (s.max == INFINITY) {
#pragma unroll
    for (int e = 0; e < kCount; ++e) s.sum += x[e] == INFINITY ? 1.f : 0.f;
    return;
  }
  float part = 0.f;
#pragma unroll
  for (int e = 0; e < kCount; ++e) part += weight_of(x[e], s.max, k);
  s.sum += part;
}
// All lanes' together, the same in every lane.
__device__ __forceinline__ Stats join(Stats s, float k) {
  Stats r = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.max = fmaxf(r.max, __shfl_xor_sync(0xffffffffu, r.max, o));
  r.sum = s.sum * weight_of_any(s.max, r.max, k);
  r.first = s.max == r.max ? s.first : 0x7fffffff;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
    r.first = min(r.first, __shfl_xor_sync(0xffffffffu, r.first, o));
  }
  return r;
}

// Eight tokens' settings as loaded: the counts and a byte each of prompt and grammar.
struct EightSettings {
  int4 a, b;
  uint32_t prompt, allowed;
  __device__ __forceinline__ void load(const RowSettings& st, int i) {
    a = b = make_int4(0, 0, 0, 0);
    if (st.counts) {
      a = __ldg(reinterpret_cast<const int4*>(st.counts + i));
      b = __ldg(reinterpret_cast<const int4*>(st.counts + i) + 1);
    }
    prompt = st.prompt ? __ldg(st.prompt + (i >> 5)) >> (i & 31) : 0u;
    allowed = st.allowed ? __ldg(st.allowed + (i >> 5)) >> (i & 31) : 0xffu;
  }
  __device__ __forceinline__ void apply(float (&x)[8], const RowSettings& st, bool penalties) const {
    if (penalties) {
      const int c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = penalised(x[e], c[e], (prompt >> e) & 1u, st);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = fmaxf(x[e], -INFINITY);  // (NaN: -inf)
      if (!((allowed >> e) & 1u)) x[e] = -INFINITY;
    }
  }
};

// kVec: rows of logits, probabilities and counts allow 16-byte accesses.
template <class In, class Out, bool kVec, class Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kBlocksPerSm)
    logits_probs_kernel(const ProbsParams p) {
  constexpr int kThreads = Shape::kThreads, kWarps = kThreads / 32, kUnroll = Shape::kUnroll;
  extern __shared__ uint32_t s_lists[];
  __shared__ Stats s_stats;  // read by the cluster
  __shared__ Stats s_warp[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / ranks;
  const int b = (int)(row / p.rows), j = (int)(row - (int64_t)b * p.rows), V = p.vocab;
  if (p.num_rows && j >= p.num_rows[b]) return;  // (every block of the cluster)
  const In* logits = static_cast<const In*>(p.logits) + row * p.logit_stride;
  Out* probs = static_cast<Out*>(p.probs) + row * p.prob_stride;
  RowSettings st;
  st.repetition = p.repetition ? p.repetition[b] : 1.f;
  st.inverse = 1.f / st.repetition;
  st.frequency = p.frequency ? p.frequency[b] : 0.f;
  st.presence = p.presence ? p.presence[b] : 0.f;
  st.counts = p.counts ? p.counts + (int64_t)b * V : nullptr;
  st.prompt = p.prompt ? p.prompt + (int64_t)b * p.words : nullptr;
  st.allowed = p.allowed ? p.allowed + row * p.words : nullptr;
  const float temperature = p.temperature ? p.temperature[b] : 1.f;
  const bool greedy = !(temperature > 0.f), penalties = p.penalties != 0;
  // (within the positive floats: 0 or infinity times a difference could be NaN)
  const float k = fminf(fmaxf(2.f * kLog2e / temperature, 0x1p-149f), 0x1.fffffep127f);
  const int lo = (int)min((int64_t)rank * p.run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + p.run, (int64_t)V);
  const int all8 = kVec ? lo + ((hi - lo) & ~7) : lo;  // tokens from here on go one by one
  Stats mine{-INFINITY, 0.f, 0x7fffffff};

  // ---- the lists: biases, and the drafts on this row's path ----
  const uint64_t on_path =
      p.tree_mask && penalties ? p.tree_mask[row] & ~1ull & (~0ull >> (64 - p.rows)) : 0;
  const int paths = __popcll(on_path), entries = p.num_biases + paths;
  int32_t* s_token = reinterpret_cast<int32_t*>(s_lists);       // [entries]
  float* s_bias = reinterpret_cast<float*>(s_token + p.num_biases + 64);  // [num_biases]
  float* s_x = s_bias + p.num_biases;                            // [entries]
  uint32_t* s_listed = reinterpret_cast<uint32_t*>(s_x + p.num_biases + 64);  // [run / 32]
  if (entries > 0) {
    for (int i = tid; i < p.num_biases; i += kThreads) {
      s_token[i] = p.bias_tokens[(int64_t)b * p.num_biases + i];
      s_bias[i] = p.biases[(int64_t)b * p.num_biases + i];
    }
    if (tid < 64 && ((on_path >> tid) & 1u))
      s_token[p.num_biases + __popcll(on_path & ((1ull << tid) - 1))] =
          p.node_tokens[(int64_t)b * p.rows + tid];
    for (int i = tid; i < p.run / 32; i += kThreads) s_listed[i] = 0u;
    __syncthreads();
    for (int e = tid; e < entries; e += kThreads) {
      const int v = s_token[e];
      if (v < lo || v >= hi) continue;
      int count = st.counts ? max(st.counts[v], 0) : 0;
      float x = as_float(logits[v]);
      for (int i = 0; i < paths; ++i) count += s_token[p.num_biases + i] == v;
      if (penalties) x = penalised(x, count, st.prompt && bit_of(st.prompt, v), st);
      for (int i = 0; i < p.num_biases; ++i)
        if (s_token[i] == v) x += s_bias[i];
      x = fmaxf(x, -INFINITY);
      if (st.allowed && !bit_of(st.allowed, v)) x = -INFINITY;
      s_x[e] = x;
      const uint32_t bit = 1u << ((v - lo) & 31);
      if (atomicOr(&s_listed[(v - lo) >> 5], bit) & bit) continue;  // its token is in the sum
      const float one[1] = {x};
      // (greedy: a thread's entries come in no order of tokens)
      if (greedy && x == mine.max && x > -INFINITY) mine.first = min(mine.first, v);
      else add_tokens(mine, one, v, greedy, k);
    }
    __syncthreads();
  }

  // ---- first pass: the row's maximum and sum ----
  Stats dense{-INFINITY, 0.f, 0x7fffffff};
  if constexpr (kVec) {
    for (int i0 = lo + 8 * tid; i0 < all8; i0 += kUnroll * 8 * kThreads) {
      Eight<In> in[kUnroll];
      EightSettings set[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * 8 * kThreads;
        if (i < all8) {
          in[u].load(logits + i);
          set[u].load(st, i);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * 8 * kThreads;
        if (i < all8) {
          float x[8];
          in[u].get(x);
          if (entries > 0) set[u].allowed &= ~(s_listed[(i - lo) >> 5] >> ((i - lo) & 31));
          set[u].apply(x, st, penalties);
          add_tokens(dense, x, i, greedy, k);
        }
      }
    }
  }
  auto one_token = [&](int i) -> float {
    float x = as_float(logits[i]);
    if (penalties)
      x = penalised(x, st.counts ? st.counts[i] : 0, st.prompt && bit_of(st.prompt, i), st);
    x = fmaxf(x, -INFINITY);
    return st.allowed && !bit_of(st.allowed, i) ? -INFINITY : x;
  };
  for (int i = all8 + tid; i < hi; i += kThreads) {
    if (entries > 0 && ((s_listed[(i - lo) >> 5] >> ((i - lo) & 31)) & 1u)) continue;
    const float one[1] = {one_token(i)};
    add_tokens(dense, one, i, greedy, k);
  }
  // the entries' and the others'
  {
    const float top = fmaxf(mine.max, dense.max);
    mine.first = min(mine.max == top ? mine.first : 0x7fffffff, dense.max == top ? dense.first : 0x7fffffff);
    mine.sum = mine.sum * weight_of_any(mine.max, top, k) + dense.sum * weight_of_any(dense.max, top, k);
    mine.max = top;
  }
  mine = join(mine, k);
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    mine = lane < kWarps ? s_warp[lane] : Stats{-INFINITY, 0.f, 0x7fffffff};
    mine = join(mine, k);
    if (lane == 0) s_stats = mine;
  }
  cluster.sync();

  // ---- all blocks': lane r looks at block r's ----
  Stats all{-INFINITY, 0.f, 0x7fffffff};
  if (lane < ranks) all = *cluster.map_shared_rank(&s_stats, lane);
  cluster.barrier_arrive();  // (nobody leaves before the others have read its numbers)
  all = join(all, k);
  // ---- second pass: exp((x - max) / t) / sum ----
  // (a row with nothing allowed has no maximum above -inf: all of it is 0)
  const bool none = !(all.max > -INFINITY), infinite = all.max == INFINITY;
  const float factor = none ? 0.f : 1.f / all.sum;
  auto value = [&](float x, int i) -> float {
    if (greedy) return i == all.first && !none ? 1.f : 0.f;
    if (none) return 0.f;
    return (infinite ? (x == INFINITY ? 1.f : 0.f) : weight_of(x, all.max, k)) * factor;
  };
  if constexpr (kVec) {
    for (int i0 = lo + 8 * tid; i0 < all8; i0 += kUnroll * 8 * kThreads) {
      Eight<In> in[kUnroll];
      EightSettings set[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * 8 * kThreads;
        if (i < all8) {
          in[u].load(logits + i);
          set[u].load(st, i);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * 8 * kThreads;
        if (i < all8) {
          float x[8];
          in[u].get(x);
          set[u].apply(x, st, penalties);
          if (greedy || none || infinite) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = value(x[e], i + e);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = weight_of(x[e], all.max, k) * factor;
          }
          Eight<Out>::store(probs + i, x);
        }
      }
    }
  }
  for (int i = all8 + tid; i < hi; i += kThreads) put(probs + i, value(one_token(i), i));
  if (entries > 0) {
    __syncthreads();  // (what was written for the listed tokens is written again)
    for (int e = tid; e < entries; e += kThreads) {
      const int v = s_token[e];
      if (v < lo || v >= hi) continue;
      put(probs + v, value(s_x[e], v));
    }
  }
  cluster.barrier_wait();
}

template <class In, class Out, bool kVec, class Shape>
cudaError_t launch_probs(const ProbsParams& p, int ranks, cudaStream_t stream) {
  const size_t bytes = p.num_biases > 0 || p.tree_mask
                           ? 4 * (size_t)(3 * p.num_biases + 2 * 64) + (size_t)p.run / 8
                           : 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.batch * p.rows * ranks));
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.dynamicSmemBytes = bytes;  // at most 18 KB
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logits_probs_kernel<In, Out, kVec, Shape>, p);
}

template <class In, class Out>
cudaError_t launch_probs(ProbsParams p, cudaStream_t stream) {
  // blocks of a row: as many as keep 2,048 tokens each; runs of whole words of the masks
  int ranks = 1;
  while (ranks < kMaxCluster && p.vocab >= 2 * ranks * 2048) ranks *= 2;
  p.run = ((p.vocab + ranks - 1) / ranks + 31) / 32 * 32;
  const bool few = (int64_t)p.batch * p.rows * ranks <= device_sm_count();
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.probs) |
                       (uintptr_t)(p.logit_stride * (int64_t)sizeof(In)) |
                       (uintptr_t)(p.prob_stride * (int64_t)sizeof(Out)) |
                       (p.counts ? reinterpret_cast<uintptr_t>(p.counts) | (uintptr_t)((int64_t)p.vocab * 4) : 0);
  if ((at & 15u) == 0)
    return few ? launch_probs<In, Out, true, Few>(p, ranks, stream)
               : launch_probs<In, Out, true, Many>(p, ranks, stream);
  return few ? launch_probs<In, Out, false, Few>(p, ranks, stream)
             : launch_probs<In, Out, false, Many>(p, ranks, stream);
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_logits_to_probs(
    const void* logits, int64_t logit_stride, int logit_dtype, void* probs, int64_t prob_stride,
    int prob_dtype, int batch, int rows, int vocab, const float* temperature,
    const int32_t* num_rows, const int32_t* node_tokens, const uint64_t* tree_mask,
    const int32_t* token_counts, const uint32_t* prompt_mask, const float* repetition,
    const float* frequency, const float* presence, const int32_t* bias_tokens, const float* biases,
    int num_biases, const uint32_t* allowed, mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || rows < 1 || vocab < 1 || num_biases < 0) return MLA_ERR_INVALID_ARG;
  for (const int dt : {logit_dtype, prob_dtype})
    if (dt != MLA_PROB_F32 && dt != MLA_PROB_BF16) return MLA_ERR_INVALID_ARG;
  if (logit_stride < vocab || prob_stride < vocab) return MLA_ERR_INVALID_ARG;
  if ((tree_mask == nullptr) != (node_tokens == nullptr)) return MLA_ERR_INVALID_ARG;
  if (tree_mask && rows > MLA_MAX_TREE_NODES) return MLA_ERR_INVALID_ARG;
  if (num_biases > 0 && (!bias_tokens || !biases) && batch > 0) return MLA_ERR_INVALID_ARG;
  if (vocab > MLA_MAX_PROBS_VOCAB || num_biases > MLA_MAX_BIASES ||
      (int64_t)batch * rows > 0x7fffffff / kMaxCluster)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0) return MLA_OK;
  if (!logits || !probs) return MLA_ERR_INVALID_ARG;
  // in place only element by element
  if (logits == probs && (logit_dtype != prob_dtype || logit_stride != prob_stride))
    return MLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (logit_dtype == MLA_PROB_F32 ? 3u : 1u)) ||
      (reinterpret_cast<uintptr_t>(probs) & (prob_dtype == MLA_PROB_F32 ? 3u : 1u)) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return MLA_ERR_INVALID_ARG;
  const void* ptrs[11] = {temperature, num_rows,  node_tokens, token_counts, prompt_mask, repetition,
                          frequency,   presence,  bias_tokens, biases,       allowed};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MLA_ERR_INVALID_ARG;
  ProbsParams p;
  p.logits = logits;
  p.logit_stride = logit_stride;
  p.probs = probs;
  p.prob_stride = prob_stride;
  p.batch = batch;
  p.rows = rows;
  p.vocab = vocab;
  p.temperature = temperature;
  p.num_rows = num_rows;
  p.node_tokens = node_tokens;
  p.tree_mask = tree_mask;
  p.counts = token_counts;
  p.prompt = prompt_mask;
  p.repetition = repetition;
  p.frequency = frequency;
  p.presence = presence;
  p.bias_tokens = bias_tokens;
  p.biases = biases;
  p.num_biases = num_biases;
  p.allowed = allowed;
  p.words = (vocab + 31) / 32;
  p.run = 0;
  // (without a penalty the counts, the prompt and the paths change nothing)
  p.penalties = repetition || frequency || presence;
  if (!p.penalties) p.counts = nullptr, p.prompt = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool in32 = logit_dtype == MLA_PROB_F32, out32 = prob_dtype == MLA_PROB_F32;
  const cudaError_t e = in32 ? (out32 ? launch_probs<float, float>(p, s)
                                      : launch_probs<float, __nv_bfloat16>(p, s))
                             : (out32 ? launch_probs<__nv_bfloat16, float>(p, s)
                                      : launch_probs<__nv_bfloat16, __nv_bfloat16>(p, s));
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
