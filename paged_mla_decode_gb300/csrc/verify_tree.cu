// verify_tree.cu -- walk down a tree of drafted tokens and sample the token behind it.
//
// "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
// custom speculative decoding ...": drafted tokens are verified in parallel without
// changing the target model's distribution. At a node the children are tried one after
// the other. With p its target row, q the drafter's that they were drawn from, and c, W
// starting at 0 and 1, what m rejected children leave of p is
//   R(x) = max(p(x) - c q(x), 0):
// child x is kept if u q(x) W < R(x) (probability min(1, R / (W q))), and a rejection adds W to c
// and makes W the sum of the new R. (In normalised terms p' = max(p - q, 0) / Z; scaled by
// the Zs so far, the products of max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0)
// fold into the one number c, so a rejection costs one pass over the vocabulary and no
// row is ever written.) Without q a child's token was certain: it is kept with R(x) / W, and
// a rejection takes it out of p, which needs no pass at all.
//
// Arithmetic as in verify_drafts.cu: weights are integers in units of 2^-60, so sums are
// exact and the index that is sampled does not depend on their order; c is rounded to
// float32 and R once more (one fused operation), where c is neither 0 nor 1; the test
// compares in double, where u q is exact.
//
// A rejection's pass reads p and q of one node, a float each a token, and the next one cannot
// begin before it: 64 requests of up to 16 nodes over 163,840 tokens take 37 us for the 157 MB
// that their passes read one after the other; one request over 131,072 tokens 10 us, latency.
//
// A request is worked by a cluster of up to eight blocks, each summing a run of the
// vocabulary. Every block walks the tree by itself, from the same numbers: the probabilities
// of all drafts are gathered at the start, a thread a node, and what a pass sums is read from
// all blocks.
#include <algorithm>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "prob_rows.cuh"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = MLA_MAX_TREE_NODES;
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct TreeParams {
  const void* target;
  int64_t target_stride;  // elements between rows
  const void* draft;      // may be null
  int64_t draft_stride;
  const int32_t* tokens;
  const uint64_t* mask;
  const float* uniforms;
  const int32_t* num_nodes;  // may be null: max_nodes each
  const int32_t* seq_lens;   // may be null
  int batch, max_nodes, vocab;
  int32_t* out_tokens;
  int32_t* path;
  int32_t* accepted;
  int32_t* seq_lens_out;  // may be null
  int32_t* token_counts;  // may be null
};

// What is left of a node's row p: max(p - c q, 0), or p without the tokens in `gone`.
template <class T>
struct Left {
  const T* p;
  const T* q;  // null while c = 0
  float c;
  const int* gone;  // in shared memory; each once
  int num_gone;
};
__device__ __forceinline__ float left_weight(float p, float q, float c) {
  return __saturatef(fmaf(-c, weight(q), weight(p)));
}
__device__ __forceinline__ void add_slices(Slices& to, float w) {
  const Slices a = slices(w), zero = slices(0.f);
#pragma unroll
  for (int j = 0; j < 3; ++j) to.s[j] += a.s[j] - zero.s[j];
}
__device__ __forceinline__ uint64_t one_weight(float w) {
  Slices one{{0, 0, 0}};
  add_slices(one, w);
  return joined(one);
}

// Sum of a lane's share of elements lo .. hi - 1 (`gone` not looked at).
template <class T, bool kVec, int kUnroll, bool kPair>
__device__ __forceinline__ uint64_t left_sum(const Left<T>& left, int lo, int hi, int lane) {
  using W = Wide<T, kVec>;
  constexpr int kTile = 32 * W::kWide;
  static_assert(kUnroll * W::kWide <= 64, "20-bit slices of 64 elements stay within 32 bits");
  uint64_t sum = 0;
  for (int i0 = lo; i0 < hi; i0 += kUnroll * kTile) {
    W pi[kUnroll], qi[kPair ? kUnroll : 1];
#pragma unroll
    for (int t = 0; t < kUnroll; ++t) {
      const int i = i0 + t * kTile + lane * W::kWide;
      pi[t].load(left.p, i, hi);
      if constexpr (kPair) qi[t].load(left.q, i, hi);
    }
    Slices part{{0, 0, 0}};
#pragma unroll
    for (int t = 0; t < kUnroll; ++t)
#pragma unroll
      for (int k = 0; k < W::kWide; ++k)
        add_slices(part, kPair ? left_weight(pi[t].get(k), qi[kPair ? t : 0].get(k), left.c)
                               : weight(pi[t].get(k)));
    sum += joined(part);
  }
  return sum;
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) verify_tree_kernel(const TreeParams p, const int run) {
  using W = Wide<T, kVec>;
  constexpr int kUnroll = kVec ? (int)sizeof(T) : 8;  // tiles of a warp in flight
  __shared__ uint64_t s_warp[kWarps];  // sums of the warps' runs
  __shared__ uint64_t s_block[2];      // of the block's, by pass; read by the cluster
  __shared__ uint64_t s_scan[kWarps];
  __shared__ int s_parent[kMaxNodes], s_tok[kMaxNodes], s_gone[kMaxNodes], s_path[kMaxNodes];
  __shared__ float s_px[kMaxNodes], s_qx[kMaxNodes], s_u[kMaxNodes];
  __shared__ int s_token;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ranks, N = p.max_nodes, V = p.vocab;
  griddep_wait();  // all earlier work in the stream is complete
  griddep_launch_dependents();
  const int n = p.num_nodes ? p.num_nodes[b] : N;
  const int L = p.seq_lens ? p.seq_lens[b] : n;
  const T* target = static_cast<const T*>(p.target) + (int64_t)b * N * p.target_stride;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + (int64_t)b * N * p.draft_stride : nullptr;
  int32_t* out = p.out_tokens + (int64_t)b * N;
  int32_t* path = p.path + (int64_t)b * N;
  if (n < 1 || n > N || L < n) {  // left out
    if (rank == 0) {
      for (int i = tid; i < N; i += kThreads) out[i] = path[i] = -1;
      if (tid == 0) {
        p.accepted[b] = -1;
        if (p.seq_lens_out) p.seq_lens_out[b] = L;
      }
    }
    return;
  }
  if (tid < n) {  // everything the walk may ask of node `tid`
    const uint64_t before = p.mask[(int64_t)b * N + tid] & ((1ull << tid) - 1);
    const int parent = 63 - __clzll((long long)before);  // -1: none
    const int x = p.tokens[(int64_t)b * N + tid];
    s_u[tid] = unit(p.uniforms[(int64_t)b * N + tid]);
    float px = 0.f, qx = 1.f;  // (outside the vocabulary: never kept)
    if (tid > 0 && parent >= 0 && x >= 0 && x < V) {
      px = weight(to_float(target[parent * p.target_stride + x]));
      if (draft) qx = weight(to_float(draft[parent * p.draft_stride + x]));
    }
    s_parent[tid] = tid > 0 ? parent : -1;
    s_tok[tid] = x;
    s_px[tid] = px;
    s_qx[tid] = qx;
  }
  if (tid == 0) s_token = -1;
  __syncthreads();

  // this warp's run of the vocabulary
  const int lo = (int)min((int64_t)(rank * kWarps + warp) * run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + run, (int64_t)V);
  Left<T> left{target, nullptr, 0.f, s_gone, 0};
  uint64_t total = 0, before = 0;  // of all blocks; of those before this one
  int passes = 0;
  auto pass = [&]() {
    uint64_t sum = left.q != nullptr ? left_sum<T, kVec, kUnroll, true>(left, lo, hi, lane)
                                     : left_sum<T, kVec, kUnroll, false>(left, lo, hi, lane);
    if (left.num_gone > 0) {
      for (int g = lane; g < left.num_gone; g += 32) {
        const int x = s_gone[g];
        if (x >= lo && x < hi) sum -= one_weight(weight(to_float(left.p[x])));
      }
    }
    sum = warp_sum(sum);
    __syncthreads();  // (the last pass's sums are no longer read)
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const uint64_t all = warp_sum(lane < kWarps ? s_warp[lane] : 0);
      if (lane == 0) s_block[passes & 1] = all;
    }
    cluster.sync();
    const uint64_t v = lane < ranks ? *cluster.map_shared_rank(&s_block[passes & 1], lane) : 0;
    total = warp_sum(v);
    before = warp_sum(lane < rank ? v : 0);
    ++passes;
  };

  // ---- the walk: every thread of every block takes the same steps ----
  int here = 0, kept = 0;
  bool rejected = false, summed = false;
  double certain_left = 1.0;  // W, without q
  for (int i = 1; i < n; ++i) {
    if (s_parent[i] != here) continue;
    const int x = s_tok[i];
    const bool in_range = x >= 0 && x < V;
    bool keep;
    float wx = 0.f;
    if (draft) {
      wx = rejected ? left_weight(s_px[i], s_qx[i], left.c) : s_px[i];
      const double w = rejected ? (double)total * 0x1p-60 : 1.0;
      keep = in_range && (double)s_u[i] * (double)s_qx[i] * w < (double)wx;
    } else {
      bool again = false;  // a rejected child's token
      for (int g = 0; g < left.num_gone; ++g) again |= s_gone[g] == x;
      wx = again ? 0.f : s_px[i];
      keep = in_range && (double)s_u[i] * certain_left < (double)wx;
      if (!keep) {
        certain_left = fmax(certain_left - (double)wx, 0.0);
        if (in_range && !again) {
          __syncthreads();  // (every thread has read the list)
          if (tid == 0) s_gone[left.num_gone] = x;
          __syncthreads();
          ++left.num_gone;
        }
      }
    }
    if (keep) {
      here = i;
      if (tid == 0) s_path[kept] = i;
      ++kept;
      left = Left<T>{target + i * p.target_stride, nullptr, 0.f, s_gone, 0};
      rejected = summed = false;
      certain_left = 1.0;
    } else {
      if (draft) {
        const double w = rejected ? (double)total * 0x1p-60 : 1.0;
        left.q = draft + here * p.draft_stride;
        left.c = (float)((double)left.c + w);
        pass();
        summed = true;
      }
      rejected = true;
    }
  }
  if (!summed) pass();
  if (total == 0 && rejected) {  // rejections that leave nothing: the target's own distribution
    left = Left<T>{left.p, nullptr, 0.f, s_gone, 0};
    pass();
  }
  // no block leaves while another may still read its sums: arrive here, wait at the end
  // (-1 unless some block finds the border: its store comes after its wait for all blocks)
  if (rank == 0) {
    __syncthreads();
    for (int i = tid; i < N; i += kThreads) {
      const int node = i < kept ? s_path[i] : -1;
      out[i] = node >= 0 ? s_tok[node] : -1;
      if (i + 1 < N) path[i + 1] = node;
      if (node >= 0 && p.token_counts)
        atomicAdd(p.token_counts + (int64_t)b * V + s_tok[node], 1);
    }
    if (tid == 0) {
      path[0] = 0;
      p.accepted[b] = kept;
      if (p.seq_lens_out) p.seq_lens_out[b] = L - n + kept + 1;
    }
    __threadfence();
  }
  cluster.sync();
  // the border: the first token whose running sum exceeds u * total, in integers
  const uint64_t at = share(s_u[0], total);
  int w = 0;
  while (w < kWarps && before + s_warp[w] <= at) before += s_warp[w++];
  if (total == 0 || at < before || w == kWarps) return;  // in another block's run
  const int run_lo = (int)min((int64_t)(rank * kWarps + w) * run, (int64_t)V);
  const int run_hi = (int)min((int64_t)run_lo + run, (int64_t)V);
  for (int i0 = run_lo; i0 < run_hi; i0 += kThreads * W::kWide) {
    const int i = i0 + tid * W::kWide;
    W pi, qi;
    pi.load(left.p, i, run_hi);
    if (left.q != nullptr) qi.load(left.q, i, run_hi);
    uint64_t mine = 0, each[W::kWide];
#pragma unroll
    for (int k = 0; k < W::kWide; ++k) {
      float wk = left.q != nullptr ? left_weight(pi.get(k), qi.get(k), left.c) : weight(pi.get(k));
      for (int g = 0; g < left.num_gone; ++g)
        if (s_gone[g] == i + k) wk = 0.f;
      each[k] = one_weight(wk);
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
    for (int k = 0; k < kWarps; ++k) all += s_scan[k];
    before += all;
    __syncthreads();
    if (at < before) break;
  }
  if (tid == 0 && s_token >= 0) {
    out[kept] = s_token;
    if (p.token_counts) atomicAdd(p.token_counts + (int64_t)b * V + s_token, 1);
  }
}

// Blocks per request: as many as keep 2,048 tokens each (as in verify_drafts.cu).
int cluster_blocks(int vocab) {
  int c = 1;
  while (c < kMaxCluster && vocab >= 2 * c * 2048) c *= 2;
  return c;
}

template <class T, bool kVec>
cudaError_t launch_verify_tree(const TreeParams& p, cudaStream_t stream) {
  const int ranks = cluster_blocks(p.vocab);
  constexpr int kTile = 32 * Wide<T, kVec>::kWide;
  const int64_t share = (int64_t)ranks * kWarps * kTile;
  const int run = (int)((p.vocab + share - 1) / share) * kTile;
  cudaLaunchAttribute attr[2];
  attr[1] = pdl_attribute();
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_tree_kernel<T, kVec>, p, run);
}

template <class T>
cudaError_t launch_verify_tree(const TreeParams& p, cudaStream_t stream) {
  // 16-byte loads where every row starts on a 16-byte boundary
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.target) | reinterpret_cast<uintptr_t>(p.draft);
  const int64_t strides = (p.target_stride | (p.draft ? p.draft_stride : 0)) * (int64_t)sizeof(T);
  return ((at | (uintptr_t)strides) & 15u) == 0 ? launch_verify_tree<T, true>(p, stream)
                                                : launch_verify_tree<T, false>(p, stream);
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_verify_tree(const void* target_probs, int64_t target_stride,
                                      const void* draft_probs, int64_t draft_stride,
                                      int prob_dtype, const int32_t* node_tokens,
                                      const uint64_t* tree_mask, const float* uniforms,
                                      const int32_t* num_nodes, const int32_t* seq_lens, int batch,
                                      int max_nodes, int vocab, int32_t* out_tokens, int32_t* path,
                                      int32_t* num_accepted, int32_t* seq_lens_out,
                                      int32_t* token_counts, mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || max_nodes < 1 || max_nodes > MLA_MAX_TREE_NODES || vocab < 1)
    return MLA_ERR_INVALID_ARG;
  if (prob_dtype != MLA_PROB_F32 && prob_dtype != MLA_PROB_BF16) return MLA_ERR_INVALID_ARG;
  if (batch > 0x7fffffff / kMaxCluster || vocab > 1 << 30) return MLA_ERR_UNSUPPORTED;
  if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return MLA_ERR_INVALID_ARG;
  if (seq_lens_out && !seq_lens) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!target_probs || !node_tokens || !tree_mask || !uniforms || !out_tokens || !path ||
      !num_accepted)
    return MLA_ERR_INVALID_ARG;
  const uintptr_t pa = prob_dtype == MLA_PROB_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs)) & pa)
    return MLA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(tree_mask) & 7u) return MLA_ERR_INVALID_ARG;
  const void* ptrs[9] = {node_tokens, uniforms,     num_nodes,    seq_lens,    out_tokens,
                         path,        num_accepted, seq_lens_out, token_counts};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MLA_ERR_INVALID_ARG;
  const TreeParams p{target_probs, target_stride, draft_probs,  draft_stride, node_tokens,
                     tree_mask,    uniforms,      num_nodes,    seq_lens,     batch,
                     max_nodes,    vocab,         out_tokens,   path,         num_accepted,
                     seq_lens_out, token_counts};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = prob_dtype == MLA_PROB_F32 ? launch_verify_tree<float>(p, s)
                                                   : launch_verify_tree<__nv_bfloat16>(p, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
