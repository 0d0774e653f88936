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
// latency bound for few.
#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

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

template <class T>
__device__ __forceinline__ float prob(const T* row, int64_t i);
template <>
__device__ __forceinline__ float prob<float>(const float* row, int64_t i) { return __ldg(row + i); }
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(const __nv_bfloat16* row, int64_t i) {
  return __bfloat162float(row[i]);
}
// A probability within [0, 1] (NaN and negative values: 0).
__device__ __forceinline__ float weight(float x) { return fminf(fmaxf(x, 0.f), 1.f); }
__device__ __forceinline__ uint64_t fixed60(float x) { return __float2ull_rz(weight(x) * 0x1p60f); }
__device__ __forceinline__ float unit(float u) { return u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f; }

// Weight of token i: p, or what a rejection leaves of it. `q` null: all of `skip`'s is lost.
template <class T>
__device__ __forceinline__ uint64_t residual(const T* p, const T* q, int skip, int i) {
  const uint64_t a = fixed60(prob(p, i));
  if (q != nullptr) {
    const uint64_t b = fixed60(prob(q, i));
    return a > b ? a - b : 0;
  }
  return i == skip ? 0 : a;
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
  __shared__ uint64_t s_sum[kVerifyWarps];
  __shared__ int s_row, s_token;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, K = p.max_drafts, V = p.vocab;
  const int drafts = p.num_drafts ? p.num_drafts[b] : K;
  const int L = p.seq_lens ? p.seq_lens[b] : 0;
  int32_t* out = p.out_tokens + (int64_t)b * (K + 1);
  if (drafts < 0 || drafts > K || L < 0) {  // left out
    for (int i = tid; i <= K; i += kVerifyThreads) out[i] = -1;
    if (tid == 0) {
      p.accepted[b] = -1;
      if (p.seq_lens_out) p.seq_lens_out[b] = L;
    }
    return;
  }
  const T* target = static_cast<const T*>(p.target) + (int64_t)b * (K + 1) * p.target_stride;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + (int64_t)b * K * p.draft_stride : nullptr;
  const float* u = p.uniforms + (int64_t)b * (K + 1);
  if (warp == 0) {
    bool ok = false;
    if (lane < drafts) {
      const int x = p.tokens[(int64_t)b * K + lane];
      if (x >= 0 && x < V) {
        const float px = weight(prob(target + lane * p.target_stride, x));
        const float qx = draft ? weight(prob(draft + lane * p.draft_stride, x)) : 1.f;
        ok = (double)unit(u[lane]) * (double)qx < (double)px;
      }
    }
    const int a = __ffs(~__ballot_sync(0xffffffffu, ok)) - 1;  // K <= 31: some lane is false
    if (lane == 0) s_row = a;
  }
  __syncthreads();
  const int a = s_row;
  const T* row = target + a * p.target_stride;
  const T* less = a < drafts && draft ? draft + a * p.draft_stride : nullptr;
  int skip = a < drafts && !draft ? p.tokens[(int64_t)b * K + a] : -1;
  // each warp sums a run of the vocabulary
  const int run = (V + kVerifyWarps - 1) / kVerifyWarps;
  const int lo = min(warp * run, V), hi = min(lo + run, V);
  uint64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;
    for (int i = lo + lane; i < hi; i += 32) sum += residual(row, less, skip, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kVerifyWarps; ++w) total += s_sum[w];
    if (total > 0 || a == drafts) break;
    less = nullptr;  // a rejection that leaves nothing: the target's own distribution
    skip = -1;
  }
  const uint64_t at = __umul64hi(__float2ull_rz(unit(u[K]) * 0x1p64f), total);
  if (tid == 0) s_token = -1;
  __syncthreads();
  uint64_t before = 0;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  if (total > 0 && before <= at && at < before + s_sum[warp]) {
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      uint64_t c = i < hi ? residual(row, less, skip, i) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + c > at);
      if (hit) {
        if (lane == 0) s_token = i0 + __ffs(hit) - 1;
        break;
      }
      before += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  __syncthreads();
  for (int i = tid; i <= K; i += kVerifyThreads)
    out[i] = i < a ? p.tokens[(int64_t)b * K + i] : i == a ? s_token : -1;
  if (tid == 0) {
    p.accepted[b] = a;
    if (p.seq_lens_out) p.seq_lens_out[b] = L - (drafts - a);
  }
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
  if (prob_dtype == MLA_PROB_F32) verify_kernel<float><<<(unsigned)batch, kVerifyThreads, 0, s>>>(p);
  else verify_kernel<__nv_bfloat16><<<(unsigned)batch, kVerifyThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
