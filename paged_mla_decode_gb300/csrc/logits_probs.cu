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
// blocks keeps it in shared memory in between (163,840 floats are 80 KB a block): each block
// makes exp(x - its own maximum) and their sum, the blocks exchange both once, and one factor
// exp(own max - max) / sum finishes its part. Tokens that a list names (biases, drafts) are
// worked out after the others, from their logits, by a thread an entry that adds up all of its
// token's entries in order: two entries of a token write the same value.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRun = 48 * 1024;  // tokens of a block: 192 KB of shared memory
static_assert((int64_t)kMaxCluster * kMaxRun >= MLA_MAX_PROBS_VOCAB, "a row fits a cluster");

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
  float repetition, frequency, presence;
  const int32_t* counts;     // of the request; may be null
  const uint32_t* prompt;    // may be null
  const uint32_t* allowed;   // of the row; may be null
};

__device__ __forceinline__ float penalised(float x, int count, bool in_prompt, const RowSettings& s) {
  if (count > 0 || in_prompt) x = x > 0.f ? x / s.repetition : x * s.repetition;
  if (count > 0) x = x - s.frequency * (float)count - s.presence;
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

struct BlockStats {
  float max, sum;
  int first;  // greedy: the lowest token with the maximum
};

// exp((x - m) / t) with k = 2 log2(e) / t >= 0 (of half the difference, which does not
// overflow); 1 at the maximum whatever k, 0 at -inf and
// beside an infinite maximum
__device__ __forceinline__ float weight_of(float x, float m, float k) {
  const float w = fast_exp2(fmaf(0.5f, x, -0.5f * m) * k);
  return x == m ? 1.f : x == -INFINITY || m == INFINITY ? 0.f : w;
}

// kVec: rows of logits, probabilities and counts allow 16-byte accesses.
template <class In, class Out, bool kVec>
__global__ void __launch_bounds__(kThreads) logits_probs_kernel(const ProbsParams p) {
  extern __shared__ __align__(16) float s_x[];  // [run], then the lists
  __shared__ BlockStats s_stats;  // read by the cluster
  __shared__ float s_red[kWarps];
  __shared__ int s_redi[kWarps];
  __shared__ int s_paths;
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
  st.frequency = p.frequency ? p.frequency[b] : 0.f;
  st.presence = p.presence ? p.presence[b] : 0.f;
  st.counts = p.counts ? p.counts + (int64_t)b * V : nullptr;
  st.prompt = p.prompt ? p.prompt + (int64_t)b * p.words : nullptr;
  st.allowed = p.allowed ? p.allowed + row * p.words : nullptr;
  const float temperature = p.temperature ? p.temperature[b] : 1.f;
  const bool greedy = !(temperature > 0.f);
  const float k = 2.f * kLog2e / temperature;
  const int lo = (int)min((int64_t)rank * p.run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + p.run, (int64_t)V);

  // ---- lists: the biases, and the drafts on this row's path ----
  int32_t* s_bias_token = reinterpret_cast<int32_t*>(s_x + p.run);
  float* s_bias = reinterpret_cast<float*>(s_bias_token + p.num_biases);
  int32_t* s_path = reinterpret_cast<int32_t*>(s_bias + p.num_biases);  // [64]
  for (int i = tid; i < p.num_biases; i += kThreads) {
    s_bias_token[i] = p.bias_tokens[(int64_t)b * p.num_biases + i];
    s_bias[i] = p.biases[(int64_t)b * p.num_biases + i];
  }
  const uint64_t on_path =
      p.tree_mask && p.penalties ? p.tree_mask[row] & ~1ull & (~0ull >> (64 - p.rows)) : 0;
  if (tid < 64 && ((on_path >> tid) & 1u))
    s_path[__popcll(on_path & ((1ull << tid) - 1))] = p.node_tokens[(int64_t)b * p.rows + tid];
  if (tid == 0) s_paths = __popcll(on_path);

  // ---- every token, without the lists ----
  const bool plain = !p.penalties;
  float top = -INFINITY;
  if constexpr (kVec) {
    constexpr int kUnroll = 2;
    for (int i0 = lo; i0 < hi; i0 += kUnroll * 8 * kThreads) {
      Eight<In> in[kUnroll];
      int4 c[kUnroll][2];
      uint32_t seen[kUnroll], ok[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + (u * kThreads + tid) * 8;
        if (i + 8 <= hi) {
          in[u].load(logits + i);
          ok[u] = st.allowed ? __ldg(st.allowed + (i >> 5)) >> (i & 31) : 0xffu;
          seen[u] = st.prompt ? __ldg(st.prompt + (i >> 5)) >> (i & 31) : 0u;
          c[u][0] = c[u][1] = make_int4(0, 0, 0, 0);
          if (st.counts) {
            c[u][0] = __ldg(reinterpret_cast<const int4*>(st.counts + i));
            c[u][1] = __ldg(reinterpret_cast<const int4*>(st.counts + i) + 1);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + (u * kThreads + tid) * 8;
        if (i + 8 <= hi) {
          float x[8];
          in[u].get(x);
          if (!plain) {
            const int cc[8] = {c[u][0].x, c[u][0].y, c[u][0].z, c[u][0].w,
                               c[u][1].x, c[u][1].y, c[u][1].z, c[u][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (cc[e] > 0 || ((seen[u] >> e) & 1u)) x[e] = penalised(x[e], cc[e], true, st);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!((ok[u] >> e) & 1u) || isnan(x[e])) x[e] = -INFINITY;
            top = fmaxf(top, x[e]);
          }
          float4* to = reinterpret_cast<float4*>(s_x + (i - lo));
          to[0] = make_float4(x[0], x[1], x[2], x[3]);
          to[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
    }
  }
  // (all of them, one by one, or the last seven)
  for (int i = (kVec ? lo + ((hi - lo) & ~7) : lo) + tid; i < hi; i += kThreads) {
    float x = as_float(logits[i]);
    if (!plain)
      x = penalised(x, st.counts ? st.counts[i] : 0, st.prompt && bit_of(st.prompt, i), st);
    if (isnan(x) || (st.allowed && !bit_of(st.allowed, i))) x = -INFINITY;
    s_x[i - lo] = x;
    top = fmaxf(top, x);
  }
  __syncthreads();

  // ---- the tokens of the lists ----
  const int paths = s_paths, entries = p.num_biases + paths;
  if (entries > 0) {
    for (int e = tid; e < entries; e += kThreads) {
      const int v = e < p.num_biases ? s_bias_token[e] : s_path[e - p.num_biases];
      if (v < lo || v >= hi) continue;
      int count = st.counts ? max(st.counts[v], 0) : 0;
      for (int i = 0; i < paths; ++i) count += s_path[i] == v;
      float x = as_float(logits[v]);
      if (!plain) x = penalised(x, count, st.prompt && bit_of(st.prompt, v), st);
      for (int i = 0; i < p.num_biases; ++i)
        if (s_bias_token[i] == v) x += s_bias[i];
      if (isnan(x) || (st.allowed && !bit_of(st.allowed, v))) x = -INFINITY;
      s_x[v - lo] = x;
    }
    __syncthreads();
    top = -INFINITY;  // (a bias may lower the maximum)
    for (int i = tid; i < hi - lo; i += kThreads) top = fmaxf(top, s_x[i]);
  }

  // ---- this block's maximum, then its exponentials and their sum ----
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_red[warp] = top;
  __syncthreads();
  top = s_red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_red[w]);
  float sum = 0.f;
  int first = 0x7fffffff;
  const int n4 = (hi - lo) >> 2;
  if (greedy) {
    for (int i = tid; i < hi - lo; i += kThreads)
      if (s_x[i] == top) first = min(first, lo + i);
  } else {
    for (int i = tid; i < n4; i += kThreads) {
      float4 x = reinterpret_cast<float4*>(s_x)[i];
      x.x = weight_of(x.x, top, k);
      x.y = weight_of(x.y, top, k);
      x.z = weight_of(x.z, top, k);
      x.w = weight_of(x.w, top, k);
      sum += (x.x + x.y) + (x.z + x.w);
      reinterpret_cast<float4*>(s_x)[i] = x;
    }
    for (int i = 4 * n4 + tid; i < hi - lo; i += kThreads) sum += s_x[i] = weight_of(s_x[i], top, k);
  }
  __syncthreads();  // (s_red has been read)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
  }
  if (lane == 0) {
    s_red[warp] = sum;
    s_redi[warp] = first;
  }
  __syncthreads();
  if (tid == 0) {
    sum = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      sum += s_red[w];
      first = min(first, s_redi[w]);
    }
    s_stats = BlockStats{top, sum, first};
  }
  cluster.sync();

  // ---- all blocks': lane r looks at block r's ----
  BlockStats mine{-INFINITY, 0.f, 0x7fffffff};
  if (lane < ranks) mine = *cluster.map_shared_rank(&s_stats, lane);
  float all = mine.max;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
  cluster.barrier_arrive();  // (nobody leaves before the others have read its numbers)
  if (greedy) {
    int at = mine.max == all && all > -INFINITY ? mine.first : 0x7fffffff;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, o));
    for (int i = lo + tid; i < hi; i += kThreads) put(probs + i, i == at ? 1.f : 0.f);
  } else {
    float total = mine.sum * weight_of(mine.max, all, k);
    if (all == -INFINITY) total = 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    // (a row with nothing allowed has no maximum above -inf: all of it is 0)
    const float factor = all > -INFINITY && top > -INFINITY ? weight_of(top, all, k) / total : 0.f;
    int from = lo;
    if constexpr (kVec) {
      for (int i = 8 * tid; i + 8 <= hi - lo; i += 8 * kThreads) {
        const float4 a = reinterpret_cast<const float4*>(s_x + i)[0];
        const float4 c = reinterpret_cast<const float4*>(s_x + i)[1];
        const float x[8] = {a.x * factor, a.y * factor, a.z * factor, a.w * factor,
                            c.x * factor, c.y * factor, c.z * factor, c.w * factor};
        Eight<Out>::store(probs + lo + i, x);
      }
      from = lo + ((hi - lo) & ~7);
    }
    for (int i = from + tid; i < hi; i += kThreads) put(probs + i, s_x[i - lo] * factor);
  }
  cluster.barrier_wait();
}

template <class In, class Out, bool kVec>
cudaError_t launch_probs(ProbsParams p, cudaStream_t stream) {
  // blocks of a row: as many as keep 2,048 tokens each; runs of whole words of the masks
  int ranks = 1;
  while (ranks < kMaxCluster && p.vocab >= 2 * ranks * 2048) ranks *= 2;
  p.run = ((p.vocab + ranks - 1) / ranks + 31) / 32 * 32;
  const int bytes = 4 * p.run + 8 * p.num_biases + 4 * 64;
  static std::atomic<int> configured[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(logits_probs_kernel<In, Out, kVec>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * kMaxRun + 8 * MLA_MAX_BIASES + 4 * 64);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(1);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.batch * p.rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logits_probs_kernel<In, Out, kVec>, p);
}

template <class In, class Out>
cudaError_t launch_probs(const ProbsParams& p, cudaStream_t stream) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.probs) |
                       (uintptr_t)(p.logit_stride * (int64_t)sizeof(In)) |
                       (uintptr_t)(p.prob_stride * (int64_t)sizeof(Out)) |
                       (p.counts ? reinterpret_cast<uintptr_t>(p.counts) | (uintptr_t)((int64_t)p.vocab * 4) : 0);
  return (at & 15u) == 0 ? launch_probs<In, Out, true>(p, stream) : launch_probs<In, Out, false>(p, stream);
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
