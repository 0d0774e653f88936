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
// A cluster of up to eight blocks works a row in two passes over its logits: the first sums
// exponentials in every thread, relative to a reference that moves only when a logit lies far above
// it, and the blocks exchange references and sums through distributed shared memory; the second
// writes exp(x - reference) / sum. (A row kept on chip in between reads half, but leaves too few
// blocks an SM to cover the exchange.) The counts are read once for several rows of a request: a
// block keeps a byte a token, which picks the token's two factors and its difference from a table.
// A row whose sum is not a positive finite number (infinities, NaNs, nothing allowed) is done again
// one token at a time, with a running maximum and every case looked at.
//
// Measured, with what crosses between L2 and the SMs (logits twice, probabilities, counts once a
// group of rows, masks; a copy of 128 float rows moves 168 MB there in 27 us, 6.2 TB/s).
// Temperature alone: 32 x 8 rows of 163,840 bf16 logits to floats 75 us (336 MB, 4.5 TB/s), to bf16
// 53 (252 MB, 4.7); 128 x 1 float rows 52 (252 MB, 4.8). Settings cost more than their bytes, in
// work for each token: the 32 x 8 rows take 94 us with penalties, 93 with biases and a grammar, 111
// with all (390 MB, 3.5 TB/s; issue slots 49% busy); the 128 x 1 rows 74 with penalties and biases
// (336 MB, 4.5 TB/s). One request's four rows of 131,072 9.5. Rows kept on chip took 1.3 times as
// long, a ring of asynchronous copies 75 us for 73. Rows that do not allow 16-byte accesses go one
// token at a time: 32 x 8 rows of 163,841 307 us with temperature alone and 462 with all, 128 x 1
// with penalties and biases 234.
//
// Roundings beyond fp32's own: exp2 is good to 2^-22, and a repetition penalty divides by its rounded
// inverse. Against 64 bits the 32 x 8 rows are off by 1.7e-7 of their norm, a plain fp32 form by 3.5e-8.
//
// Tokens that a list names (biases, drafts) are left out of the passes, by a bit each, and
// worked out by a thread an entry, which adds up all of its token's entries in order.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
// Shapes of block. With few rows a block has an SM to itself and all of its loads should be in
// flight at once; with many, several smaller blocks an SM cover each other's waits.
struct Few {
  static constexpr int kThreads = 1024, kBlocksPerSm = 1, kUnroll = 2;
};
struct Many {
  static constexpr int kThreads = 256, kBlocksPerSm = 4, kUnroll = 1;
};
constexpr int kMaxGroup = 8;  // rows of a block, one after the other

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
  int group;  // rows of a block
  int penalties;
};

// What changes a request's logits, the same for all of its tokens.
struct RowSettings {
  float repetition, inverse, frequency, presence;
  const int32_t* counts;     // of the request; may be null
  const uint32_t* prompt;    // may be null
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

// A reference and the sum of exp((x - ref) / t): ref the maximum, or in the fast pass
// something within 2^kSlack of it. Greedy: the maximum, and the lowest token with it.
struct Stats {
  float ref, sum;
  int first;
};
constexpr float kSlack = 60.f;       // (a sum of 2^19 terms up to 2^60 is far from overflow)
constexpr float kNoRef = -3.0e38f;   // before any token (weights relative to it are 0)

// exp((x - m) / t) for any x and m, with k = 2 log2(e) / t (of half the difference, which does
// not overflow); beside an infinite maximum only its equals have a weight
__device__ __forceinline__ float weight_of_any(float x, float m, float k) {
  if (x == m) return m > -INFINITY ? 1.f : 0.f;
  return m == INFINITY || x == -INFINITY ? 0.f : fast_exp2(fmaf(0.5f, x, -0.5f * m) * k);
}
// One token, every case looked at (x is no NaN).
__device__ __forceinline__ void add_careful(Stats& s, float x, int token, bool greedy, float k) {
  if (x > s.ref) {
    s.sum *= weight_of_any(s.ref, x, k);
    s.ref = x;
    s.first = token;
  } else if (x == s.ref && x > -INFINITY) {
    s.first = min(s.first, token);
  }
  if (!greedy) s.sum += weight_of_any(x, s.ref, k);
}
// Tokens of finite logits (or -inf), k1 = log2(e) / t, slack = kSlack / k1.
template <int kCount>
__device__ __forceinline__ void add_fast(Stats& s, const float (&x)[kCount], float k1, float slack) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < kCount; ++e) top = fmaxf(top, x[e]);
  if (top > s.ref + slack) {
    s.sum *= fast_exp2((s.ref - top) * k1);
    s.ref = top;
  }
  if constexpr (kCount == 1) {
    s.sum += fast_exp2((x[0] - s.ref) * k1);
  } else {
    const float2 r2 = make_float2(-s.ref, -s.ref), k2 = make_float2(k1, k1);
    float2 part = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < kCount; e += 2) {
      const float2 d = mul2(add2(make_float2(x[e], x[e + 1]), r2), k2);
      part = add2(part, make_float2(fast_exp2(d.x), fast_exp2(d.y)));
    }
    s.sum += part.x + part.y;
  }
}
template <int kCount>
__device__ __forceinline__ void add_greedy(Stats& s, const float (&x)[kCount], int token) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < kCount; ++e) top = fmaxf(top, x[e]);
  if (top > s.ref) {
    s.ref = top;
#pragma unroll
    for (int e = kCount - 1; e >= 0; --e)
      if (x[e] == top) s.first = token + e;
  }
}
// All lanes' together, the same in every lane.
__device__ __forceinline__ Stats join(const Stats& s, float k) {
  Stats r = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.ref = fmaxf(r.ref, __shfl_xor_sync(0xffffffffu, r.ref, o));
  r.sum = s.sum * weight_of_any(s.ref, r.ref, k);
  r.first = s.ref == r.ref ? s.first : 0x7fffffff;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.sum += __shfl_xor_sync(0xffffffffu, r.sum, o);
    r.first = min(r.first, __shfl_xor_sync(0xffffffffu, r.first, o));
  }
  return r;
}

__device__ __forceinline__ uint32_t byte_of(const uint32_t* words, int i) {  // i: a multiple of 8
  return (__ldg(words + (i >> 5)) >> (i & 31)) & 0xffu;
}
// A token's byte: 0 not seen, 1 in the prompt only, count + 1 up to 254, 255 beyond. By byte, a
// table holds what it makes of a logit: x (x > 0 ? up : down) - off, as (up, down, off).
constexpr uint32_t kCodeBeyond = 255;
__device__ __forceinline__ uint2 codes_of(const int32_t* counts, const uint32_t* prompt, int i) {
  uint32_t seen = prompt ? byte_of(prompt, i) : 0u, w[2] = {0, 0};
  int4 a = make_int4(0, 0, 0, 0), b = a;
  if (counts) {
    a = __ldg(reinterpret_cast<const int4*>(counts + i));
    b = __ldg(reinterpret_cast<const int4*>(counts + i) + 1);
  }
  if (seen != 0 || (a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) != 0) {
    const int n[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t code = n[e] > 0 ? min((uint32_t)n[e] + 1u, kCodeBeyond) : (seen >> e) & 1u;
      w[e >> 2] |= code << (8 * (e & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void apply_codes(float (&x)[8], const uint2& codes, const float4* table,
                                            const int32_t* counts, int i, const RowSettings& st) {
  if ((codes.x | codes.y) == 0) return;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint32_t w = e < 4 ? codes.x : codes.y;
    const float4 a = table[(w >> (8 * (e & 3))) & 0xffu], b = table[(w >> (8 * (e & 3) + 8)) & 0xffu];
    const float2 f = make_float2(x[e] > 0.f ? a.x : a.y, x[e + 1] > 0.f ? b.x : b.y);
    const float2 v = add2(mul2(make_float2(x[e], x[e + 1]), f), make_float2(-a.z, -b.z));
    x[e] = v.x;
    x[e + 1] = v.y;
  }
  // (the table takes a count beyond it as 0: the rest of its difference)
  if (((~codes.x - 0x01010101u) & codes.x & 0x80808080u) | ((~codes.y - 0x01010101u) & codes.y & 0x80808080u)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t code = ((e < 4 ? codes.x : codes.y) >> (8 * (e & 3))) & 0xffu;
      if (code == kCodeBeyond) x[e] -= fmaf(st.frequency, (float)counts[i + e], st.presence);
    }
  }
}
// Tokens whose bit is not set: -inf.
__device__ __forceinline__ void hide(float (&x)[8], uint32_t bits) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (!((bits >> e) & 1u)) x[e] = -INFINITY;
}

// A token that a bias or a draft names.
struct Special {
  uint64_t nodes;  // the drafts that are this token
  int token;       // -1: another run's, or an earlier entry's
  int count;       // without the drafts on a row's path
  float bias;
  int in_prompt;
};

// kVec: rows of logits, probabilities and counts allow 16-byte accesses. (Without, every row goes
// the careful way.) kPen: there are penalties.
template <class In, class Out, bool kVec, bool kPen, class Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kBlocksPerSm)
    logits_probs_kernel(const ProbsParams p) {
  constexpr int kThreads = Shape::kThreads, kWarps = kThreads / 32, kUnroll = Shape::kUnroll;
  extern __shared__ __align__(16) uint8_t s_all[];
  __shared__ Stats s_stats[2];  // by exchange; read by the cluster
  __shared__ Stats s_warp[kWarps];
  __shared__ float4 s_table[kPen ? 256 : 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (p.rows + p.group - 1) / p.group;  // of a request
  const int unit = blockIdx.x / ranks;
  const int b = unit / groups, j0 = (unit - b * groups) * p.group, V = p.vocab;
  griddep_wait();  // all earlier work in the stream is complete
  griddep_launch_dependents();
  const int j1 = min(j0 + p.group, p.num_rows ? min(p.num_rows[b], p.rows) : p.rows);
  if (j0 >= j1) return;  // (every block of the cluster)
  RowSettings st;
  st.repetition = kPen && p.repetition ? p.repetition[b] : 1.f;
  st.inverse = 1.f / st.repetition;
  st.frequency = kPen && p.frequency ? p.frequency[b] : 0.f;
  st.presence = kPen && p.presence ? p.presence[b] : 0.f;
  st.counts = kPen && p.counts ? p.counts + (int64_t)b * V : nullptr;
  st.prompt = kPen && p.prompt ? p.prompt + (int64_t)b * p.words : nullptr;
  const float temperature = p.temperature ? p.temperature[b] : 1.f;
  const bool greedy = !(temperature > 0.f);
  // (within the positive floats: 0 or infinity times a difference could be NaN)
  const float k = fminf(fmaxf(2.f * kLog2e / temperature, 0x1p-149f), 0x1.fffffep127f);
  const float k1 = 0.5f * k, slack = kSlack / k1;
  const int lo = (int)min((int64_t)rank * p.run, (int64_t)V);
  const int hi = (int)min((int64_t)lo + p.run, (int64_t)V);
  const int all8 = kVec ? lo + ((hi - lo) & ~7) : lo;  // tokens from here on go one by one
  const int64_t row0 = (int64_t)b * p.rows;
  // the run's bytes, written and read by the thread that has the tokens; then the lists
  uint2* s_codes = reinterpret_cast<uint2*>(s_all);
  uint8_t* s_lists = s_all + (kVec && kPen ? p.run : 0);
  if constexpr (kPen && kVec) {
    for (int c = tid; c < 256; c += kThreads) {
      const bool counted = c > 1 && c < (int)kCodeBeyond;
      s_table[c] = c == 0 ? make_float4(1.f, 1.f, 0.f, 0.f)
                          : make_float4(st.inverse, st.repetition,
                                        counted ? fmaf(st.frequency, (float)(c - 1), st.presence) : 0.f, 0.f);
    }
    __syncthreads();
  }

  // ---- the lists: biases and drafts ----
  const int nodes = kPen && p.tree_mask ? p.rows : 0;  // (<= 64)
  const int specials = p.num_biases + nodes;
  Special* s_special = reinterpret_cast<Special*>(s_lists);                        // [specials]
  float* s_special_x = reinterpret_cast<float*>(s_special + p.num_biases + 64);    // [specials], of the row
  uint32_t* s_listed = reinterpret_cast<uint32_t*>(s_special_x + p.num_biases + 64);  // [run / 32]
  int32_t* s_bias_token = reinterpret_cast<int32_t*>(s_listed + p.run / 32);       // [specials]
  float* s_bias = reinterpret_cast<float*>(s_bias_token + p.num_biases + 64);      // [num_biases]
  if (specials > 0) {
    for (int i = tid; i < p.num_biases; i += kThreads) {
      s_bias_token[i] = p.bias_tokens[(int64_t)b * p.num_biases + i];
      s_bias[i] = p.biases[(int64_t)b * p.num_biases + i];
    }
    if (tid < nodes)  // (node 0's token is among the counted)
      s_bias_token[p.num_biases + tid] = tid > 0 ? p.node_tokens[row0 + tid] : -1;
    for (int i = tid; i < p.run / 32; i += kThreads) s_listed[i] = 0u;
    __syncthreads();
    for (int e = tid; e < specials; e += kThreads) {
      const int v = s_bias_token[e];
      Special t{0, -1, 0, 0.f, 0};
      if (v >= lo && v < hi) {
        int entry = specials;  // the first one of this token
        for (int i = specials - 1; i >= p.num_biases; --i)
          if (s_bias_token[i] == v) t.nodes |= 1ull << (i - p.num_biases), entry = i;
        for (int i = p.num_biases - 1; i >= 0; --i)
          if (s_bias_token[i] == v) entry = i;
        if (entry == e) {
          t.token = v;
          t.count = st.counts ? max(st.counts[v], 0) : 0;
          t.in_prompt = st.prompt ? bit_of(st.prompt, v) : 0;
          for (int i = e; i < p.num_biases; ++i)
            if (s_bias_token[i] == v) t.bias += s_bias[i];
          atomicOr(&s_listed[(v - lo) >> 5], 1u << ((v - lo) & 31));
        }
      }
      s_special[e] = t;
    }
    __syncthreads();
  }
  auto listed8 = [&](int i) -> uint32_t { return s_listed[(i - lo) >> 5] >> ((i - lo) & 31); };

  int exchanges = 0;
  for (int j = j0; j < j1; ++j) {
    const In* logits = static_cast<const In*>(p.logits) + (row0 + j) * p.logit_stride;
    Out* probs = static_cast<Out*>(p.probs) + (row0 + j) * p.prob_stride;
    const uint32_t* allowed = p.allowed ? p.allowed + (row0 + j) * p.words : nullptr;
    auto final_of = [&](float x, int v) -> float {  // (NaN: -inf)
      return allowed && !bit_of(allowed, v) ? -INFINITY : fmaxf(x, -INFINITY);
    };
    if (specials > 0) {  // their logits with everything, each read back by the thread that wrote it
      const uint64_t on_path = nodes > 0 ? p.tree_mask[row0 + j] : 0;
      for (int e = tid; e < specials; e += kThreads) {
        const Special t = s_special[e];
        if (t.token < 0) continue;
        float x = as_float(logits[t.token]);
        if (kPen) x = penalised(x, t.count + __popcll(t.nodes & on_path), t.in_prompt, st);
        s_special_x[e] = final_of(x + t.bias, t.token);
      }
    }
    auto each_listed = [&](auto use) {
      for (int e = tid; e < specials; e += kThreads)
        if (s_special[e].token >= 0) use(s_special_x[e], s_special[e].token);
    };
    auto one_token = [&](int i) -> float {
      float x = as_float(logits[i]);
      if (kPen)
        x = penalised(x, st.counts ? st.counts[i] : 0, st.prompt && bit_of(st.prompt, i), st);
      return final_of(x, i);
    };
    // a thread's tokens by eights, to `use(x, i)`; `apart`: without the listed; `fresh`: the
    // first time for this request, when their bytes are made
    auto each8 = [&](bool apart, bool fresh, auto use) {
      if constexpr (kVec) {
        for (int i0 = lo + 8 * tid; i0 < all8; i0 += kUnroll * 8 * kThreads) {
          Eight<In> in[kUnroll];
          uint32_t bits[kUnroll];
          [[maybe_unused]] uint2 codes[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * 8 * kThreads;
            if (u == 0 || i < all8) {
              in[u].load(logits + i);
              bits[u] = allowed ? byte_of(allowed, i) : 0xffu;
            }
          }
          if constexpr (kPen) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
              const int i = i0 + u * 8 * kThreads;
              if (u == 0 || i < all8)
                codes[u] = fresh ? codes_of(st.counts, st.prompt, i) : s_codes[(i - lo) >> 3];
            }
          }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * 8 * kThreads;
            if (u == 0 || i < all8) {
              float x[8];
              in[u].get(x);
              if constexpr (kPen) {
                if (fresh) s_codes[(i - lo) >> 3] = codes[u];
                apply_codes(x, codes[u], s_table, st.counts, i, st);
              }
              if (allowed || apart) hide(x, apart ? bits[u] & ~listed8(i) : bits[u]);
              use(x, i);
            }
          }
        }
      }
    };

  Stats mine, all;
    // the blocks' numbers together: lane r looks at block r's
    auto exchange = [&]() {
      mine = join(mine, k);
      __syncthreads();  // (the last exchange's have been read)
      if (lane == 0) s_warp[warp] = mine;
      __syncthreads();
      if (warp == 0) {
        Stats r = lane < kWarps ? s_warp[lane] : Stats{-INFINITY, 0.f, 0x7fffffff};
        r = join(r, k);
        if (lane == 0) s_stats[exchanges & 1] = r;
      }
      // (the numbers of two exchanges ago were read before the last such barrier)
      cluster.sync();
      all = Stats{-INFINITY, 0.f, 0x7fffffff};
      if (lane < ranks) all = *cluster.map_shared_rank(&s_stats[exchanges & 1], lane);
      all = join(all, k);
      ++exchanges;
    };

    // ---- first pass ----
    bool careful = !kVec || greedy || k1 < 0x1p-60f;
    const bool fresh = j == j0;
    if (!careful) {
      mine = Stats{kNoRef, 0.f, 0};
      each8(specials > 0, fresh, [&](const float(&x)[8], int) { add_fast(mine, x, k1, slack); });
      auto add = [&](float x, int) {
        const float one[1] = {x};
        add_fast(mine, one, k1, slack);
      };
      for (int i = all8 + tid; i < hi; i += kThreads)
        if (specials == 0 || !(listed8(i) & 1u)) add(one_token(i), i);
      if (specials > 0) each_listed(add);
      exchange();
      careful = !(all.sum > 0.f && all.sum < INFINITY);
    }
    if (careful) {
      mine = Stats{-INFINITY, 0.f, 0x7fffffff};
      if (greedy) each8(specials > 0, fresh, [&](const float(&x)[8], int i) { add_greedy(mine, x, i); });
      for (int i = (greedy ? all8 : lo) + tid; i < hi; i += kThreads)
        if (specials == 0 || !(listed8(i) & 1u)) add_careful(mine, one_token(i), i, greedy, k);
      if (specials > 0) each_listed([&](float x, int v) { add_careful(mine, x, v, greedy, k); });
      exchange();
    }

    // ---- second pass: exp((x - ref) / t) / sum ----
    // (a row with nothing allowed has no reference above -inf: all of it is 0)
    const bool none = !(all.ref > -INFINITY);
    const float factor = none ? 0.f : 1.f / all.sum;
    auto value = [&](float x, int i) -> float {
      if (greedy) return i == all.first && !none ? 1.f : 0.f;
      if (!careful) return fast_exp2((x - all.ref) * k1) * factor;
      return none ? 0.f : weight_of_any(x, all.ref, k) * factor;
    };
    if (!careful) {
      const float2 k2 = make_float2(k1, k1), r2 = make_float2(-all.ref, -all.ref), f2 = make_float2(factor, factor);
      each8(false, false, [&](float(&x)[8], int i) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 d = mul2(add2(make_float2(x[e], x[e + 1]), r2), k2);
          const float2 w = mul2(make_float2(fast_exp2(d.x), fast_exp2(d.y)), f2);
          x[e] = w.x;
          x[e + 1] = w.y;
        }
        Eight<Out>::store(probs + i, x);
      });
    } else if (kVec && greedy) {
      for (int i = lo + 8 * tid; i < all8; i += 8 * kThreads) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = value(0.f, i + e);
        Eight<Out>::store(probs + i, x);
      }
    }
    for (int i = (!careful || greedy ? all8 : lo) + tid; i < hi; i += kThreads)
      put(probs + i, value(greedy ? 0.f : one_token(i), i));
    if (specials > 0 && !greedy) {
      __syncthreads();  // (what was written for the listed tokens is written again)
      each_listed([&](float x, int v) { put(probs + v, value(x, v)); });
    }
  }
  cluster.sync();  // nobody leaves before the others have read its numbers
}

template <class In, class Out, bool kVec, bool kPen, class Shape>
cudaError_t launch_probs(const ProbsParams& p, int ranks, cudaStream_t stream) {
  const size_t entries = (size_t)p.num_biases + 64;
  const size_t bytes = (kVec && kPen ? p.run : 0) +
                       (p.num_biases > 0 || (kPen && p.tree_mask)
                            ? (sizeof(Special) + 12) * entries + (size_t)p.run / 8
                            : 0);
  if (bytes > 40 * 1024) {
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev].load()) {
      const cudaError_t e = cudaFuncSetAttribute(logits_probs_kernel<In, Out, kVec, kPen, Shape>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) configured[dev].store(1);
    }
  }
  cudaLaunchAttribute attr[2];
  attr[1] = pdl_attribute();
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.batch * ((p.rows + p.group - 1) / p.group) * ranks));
  cfg.blockDim = dim3(Shape::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logits_probs_kernel<In, Out, kVec, kPen, Shape>, p);
}

template <class In, class Out>
cudaError_t launch_probs(ProbsParams p, cudaStream_t stream) {
  // blocks of a row: as many as keep 2,048 tokens each; runs of whole words of the masks
  int ranks = 1;
  while (ranks < kMaxCluster && p.vocab >= 2 * ranks * 2048) ranks *= 2;
  p.run = ((p.vocab + ranks - 1) / ranks + 31) / 32 * 32;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) | reinterpret_cast<uintptr_t>(p.probs) |
                       (uintptr_t)(p.logit_stride * (int64_t)sizeof(In)) |
                       (uintptr_t)(p.prob_stride * (int64_t)sizeof(Out)) |
                       (p.counts ? reinterpret_cast<uintptr_t>(p.counts) | (uintptr_t)((int64_t)p.vocab * 4) : 0);
  const int64_t blocks = (int64_t)p.batch * p.rows * ranks;
  const int sms = device_sm_count();
  // rows that share their request's counts, as long as that leaves several blocks an SM
  p.group = p.counts || p.prompt ? (int)std::min<int64_t>(std::max<int64_t>(blocks / (3 * sms), 1), kMaxGroup) : 1;
  p.group = std::min(p.group, p.rows);
  if ((at & 15u) != 0) return launch_probs<In, Out, false, true, Many>(p, ranks, stream);
  if (blocks <= sms)
    return p.penalties ? launch_probs<In, Out, true, true, Few>(p, ranks, stream)
                       : launch_probs<In, Out, true, false, Few>(p, ranks, stream);
  return p.penalties ? launch_probs<In, Out, true, true, Many>(p, ranks, stream)
                     : launch_probs<In, Out, true, false, Many>(p, ranks, stream);
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
  p.run = p.group = 0;
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
