// kv_alloc.cu -- extend requests by new tokens: pages, block-table rows, page tags, slots.
//
// The page allocator's side of a step over one physical paged cache ("Smaller, faster,
// safer: running Kimi and GLM at scale", section "Protecting a shared KV cache": a page's
// tag changes whenever the page is handed out again, and each request keeps the tags its
// pages had when it was given them), computed on the device from the requests' lengths,
// so that a captured step needs no host copy of them.
//
//   rows:   cu[b + 1] = cu[b] + n_b                       (a running sum over requests)
//   need_b  = max(0, ceil((L_b + n_b) / 64) - held_b)     (0 for a refused request)
//   first_b = running sum of need: request b takes free_pages[count - 1 - first_b - k]
//
// Two running sums over the batch and 4 bytes per new token: latency bound. One block
// scans the requests in chunks of its size; each chunk's pages and slots are then spread
// over the threads, which find their request by bisection in shared memory.
#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kAllocThreads = 1024;
constexpr int kAllocWarps = kAllocThreads / 32;

struct AllocParams {
  const int32_t* seq_lens;
  const int32_t* new_tokens;
  int batch;
  const int32_t* held;
  const int32_t* free_pages;
  const int32_t* free_count;
  int64_t free_capacity;
  int64_t num_pages;
  int32_t* block_table;
  int max_pages;
  uint32_t* page_tags;
  uint32_t* expected_tags;
  int32_t* seq_lens_out;
  int32_t* held_out;
  int32_t* free_count_out;
  int32_t* cu;
  int32_t* slots;
  int64_t num_slots;
  uint32_t* status;
};

struct AllocShared {
  int64_t warp_sum[kAllocWarps];
  int64_t row_end[kAllocThreads];   // rows of the chunk's requests, ends
  int64_t page_end[kAllocThreads];  // their pages, ends
  int32_t len[kAllocThreads];       // cached tokens; -1: refused
  int32_t held[kAllocThreads];
};

// Inclusive running sum over the block's threads; every thread gets its own and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < kAllocWarps ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane < kAllocWarps) warp_sum[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += warp_sum[warp - 1];
  *total = warp_sum[kAllocWarps - 1];
  __syncthreads();
  return v;
}

// First i < n with end[i] > x (n if there is none).
__device__ __forceinline__ int first_after(const int64_t* end, int n, int64_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int64_t pages_for(int64_t tokens) {
  return (tokens + kPageSize - 1) / kPageSize;
}

__global__ void __launch_bounds__(kAllocThreads) kv_alloc_kernel(const AllocParams p) {
  __shared__ AllocShared sm;
  const int tid = threadIdx.x;
  const int64_t count = min(max((int64_t)p.free_count[0], (int64_t)0), p.free_capacity);
  int64_t row0 = 0, page0 = 0, taken = 0;  // rows, pages asked for and pages taken so far
  for (int b0 = 0; b0 < p.batch; b0 += kAllocThreads) {
    const int b = b0 + tid;
    const bool live = b < p.batch;
    const int L = live ? p.seq_lens[b] : 0, held = live ? p.held[b] : 0;
    const int asked = live ? p.new_tokens[b] : 0;
    const int64_t n = max(asked, 0);
    int64_t rows, pages;
    const int64_t row_end = row0 + block_scan(n, sm.warp_sum, &rows);
    uint32_t st = 0;
    if (L < 0 || asked < 0 || held < 0 || held > p.max_pages || pages_for(L) > held)
      st = MLA_KV_ALLOC_BAD_LENGTH;
    else if (pages_for(L + n) > p.max_pages) st = MLA_KV_ALLOC_TABLE_FULL;
    else if (row_end > p.num_slots) st = MLA_KV_ALLOC_SLOTS_FULL;
    const int64_t need = live && st == 0 ? max(pages_for(L + n) - held, (int64_t)0) : 0;
    const int64_t page_end = page0 + block_scan(need, sm.warp_sum, &pages);
    if (need > 0 && page_end > count) st = MLA_KV_ALLOC_NO_PAGES;
    const bool grown = need > 0 && st == 0;
    sm.row_end[tid] = row_end;
    sm.page_end[tid] = page_end;
    sm.len[tid] = st == 0 ? L : -1;
    sm.held[tid] = held;
    if (live) {
      p.seq_lens_out[b] = st == 0 ? (int32_t)(L + n) : -1;
      p.held_out[b] = held + (grown ? (int32_t)need : 0);
      p.status[b] = st;
      p.cu[b + 1] = (int32_t)min(row_end, (int64_t)0x7fffffff);
    }
    // the requests that got pages are a prefix of those that asked: the page count only grows
    int64_t got = grown ? page_end : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) got = max(got, __shfl_xor_sync(0xffffffffu, got, o));
    if ((tid & 31) == 0) sm.warp_sum[tid >> 5] = got;
    __syncthreads();
    for (int w = 0; w < kAllocWarps; ++w) taken = max(taken, sm.warp_sum[w]);
    const int nb = min(kAllocThreads, p.batch - b0);
    // pages: from page0 up to what was taken
    for (int64_t x = page0 + tid; x < min(page0 + pages, taken); x += kAllocThreads) {
      const int i = first_after(sm.page_end, nb, x);
      const int64_t k = x - (i > 0 ? sm.page_end[i - 1] : page0);
      const int64_t at = (int64_t)(b0 + i) * p.max_pages + sm.held[i] + k;
      const int32_t page = p.free_pages[count - 1 - x];
      p.block_table[at] = page;
      if (p.page_tags != nullptr && page >= 0 && page < p.num_pages) {
        const uint32_t tag = p.page_tags[page] + 1;
        p.page_tags[page] = tag;
        p.expected_tags[at] = tag;
      }
    }
    // slots: pages that the request held already come from its row, the new ones from the
    // free list, so that no thread waits for another's table entry
    for (int64_t x = row0 + tid; x < min(row0 + rows, p.num_slots); x += kAllocThreads) {
      const int i = first_after(sm.row_end, nb, x);
      int64_t slot = -1;
      if (sm.len[i] >= 0) {
        const int64_t pos = sm.len[i] + x - (i > 0 ? sm.row_end[i - 1] : row0);
        const int64_t j = pos / kPageSize;
        const int32_t page =
            j < sm.held[i]
                ? p.block_table[(int64_t)(b0 + i) * p.max_pages + j]
                : p.free_pages[count - 1 - (i > 0 ? sm.page_end[i - 1] : page0) - (j - sm.held[i])];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * kPageSize + pos % kPageSize;
      }
      p.slots[x] = (int32_t)slot;
    }
    row0 += rows;
    page0 += pages;
    __syncthreads();
  }
  for (int64_t x = row0 + tid; x < p.num_slots; x += kAllocThreads) p.slots[x] = -1;
  if (tid == 0) {
    p.cu[0] = 0;
    p.free_count_out[0] = (int32_t)(count - taken);
  }
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_kv_alloc(const int32_t* seq_lens, const int32_t* new_tokens, int batch,
                                   int page_size, const int32_t* pages_held,
                                   const int32_t* free_pages, const int32_t* free_count,
                                   int64_t free_capacity, int64_t num_pages, int32_t* block_table,
                                   int max_pages, uint32_t* page_tags, uint32_t* expected_tags,
                                   int32_t* seq_lens_out, int32_t* pages_held_out,
                                   int32_t* free_count_out, int32_t* cu_tokens,
                                   int32_t* slot_mapping, int64_t num_slots,
                                   uint32_t* request_status, mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || free_capacity < 0 || num_pages < 0 || max_pages < 1 || num_slots < 0)
    return MLA_ERR_INVALID_ARG;
  if (page_size != kPageSize) return MLA_ERR_UNSUPPORTED;
  if (num_pages > 0x7fffffff / kPageSize || num_slots > 0x7fffffffLL ||
      max_pages > 0x7fffffff / kPageSize)
    return MLA_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !cu_tokens) return MLA_ERR_INVALID_ARG;
  if (batch > 0 && (!seq_lens || !new_tokens || !pages_held || !block_table || !seq_lens_out ||
                    !pages_held_out || !request_status))
    return MLA_ERR_INVALID_ARG;
  if ((free_capacity > 0 && !free_pages) || (num_slots > 0 && !slot_mapping))
    return MLA_ERR_INVALID_ARG;
  if ((page_tags == nullptr) != (expected_tags == nullptr)) return MLA_ERR_INVALID_ARG;
  const void* ptrs[14] = {seq_lens,      new_tokens,   pages_held,     free_pages,     free_count,
                          block_table,   page_tags,    expected_tags,  seq_lens_out,   pages_held_out,
                          free_count_out, cu_tokens,   slot_mapping,   request_status};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MLA_ERR_INVALID_ARG;
  const AllocParams p{seq_lens,  new_tokens,    batch,         pages_held,   free_pages,
                      free_count, free_capacity, num_pages,    block_table,  max_pages,
                      page_tags, expected_tags, seq_lens_out,  pages_held_out, free_count_out,
                      cu_tokens, slot_mapping,  num_slots,     request_status};
  kv_alloc_kernel<<<1, kAllocThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
