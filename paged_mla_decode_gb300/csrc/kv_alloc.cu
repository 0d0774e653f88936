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
// Two running sums over the batch and 4 bytes written per new token: latency bound for a
// step's few tokens, then bound by the slots' stores. Every block scans the requests, in
// chunks of its size, and fills its own run of rows (a thread finds its request by
// bisection in shared memory, once per 128 rows); the row of a new page's first token
// also writes the page's table entry and tag. The page ids of new pages come from the
// free list itself, so that no row waits for another's table entry.
#include <algorithm>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kAllocThreads = 1024;    // at most; a step's few rows take fewer
constexpr int kAllocWarps = kAllocThreads / 32;
constexpr int64_t kBlockRows = 4096;   // rows that are worth a block of their own

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

// Inclusive running sums of two values over the block's threads, in place; every thread
// also gets the totals.
struct Pair {
  int64_t x, y;
};
__device__ __forceinline__ Pair block_scan(Pair& v, Pair* warp_sum, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, v.x, o), b = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) v.x += a, v.y += b;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums
  Pair s = lane < warps ? warp_sum[lane] : Pair{0, 0};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, s.x, o), b = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) s.x += a, s.y += b;
  }
  const int64_t px = __shfl_sync(0xffffffffu, s.x, max(warp - 1, 0));
  const int64_t py = __shfl_sync(0xffffffffu, s.y, max(warp - 1, 0));
  if (warp > 0) v.x += px, v.y += py;
  const Pair total{__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31)};
  __syncthreads();  // the sums are no longer read
  return total;
}

struct AllocShared {
  Pair warp_sum[kAllocWarps];
  int64_t row_end[kAllocThreads];     // rows of the chunk's requests, ends
  int64_t first_page[kAllocThreads];  // pages taken before each
  int32_t len[kAllocThreads];         // cached tokens; -1: refused
  int32_t held[kAllocThreads];
};

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

// kFill: rows [blockIdx.x * rows_per, + rows_per) of the slot map, with the new pages that
// begin there. kCommit: block 0 writes the per-request outputs, which may be the inputs:
// then no other block may still read them (one block in all, or a launch of its own).
template <bool kFill, bool kCommit>
__global__ void __launch_bounds__(kAllocThreads)
    kv_alloc_kernel(const AllocParams p, const int64_t rows_per, const int warp_rows) {
  __shared__ AllocShared sm;
  const int threads = blockDim.x, warps = threads >> 5;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool commit = kCommit && blockIdx.x == 0;
  const int64_t lo = blockIdx.x * rows_per, hi = min(lo + rows_per, p.num_slots);
  const int64_t count = min(max((int64_t)p.free_count[0], (int64_t)0), p.free_capacity);
  int64_t row0 = 0, page0 = 0, taken = 0;  // rows, pages asked for and pages taken so far
  for (int b0 = 0; b0 < p.batch; b0 += threads) {
    const int b = b0 + tid;
    const bool live = b < p.batch;
    const int L = live ? p.seq_lens[b] : 0, held = live ? p.held[b] : 0;
    const int asked = live ? p.new_tokens[b] : 0;
    const int64_t n = max(asked, 0);
    uint32_t st = 0;
    if (L < 0 || asked < 0 || held < 0 || held > p.max_pages || pages_for(L) > held)
      st = MLA_KV_ALLOC_BAD_LENGTH;
    else if (pages_for(L + n) > p.max_pages) st = MLA_KV_ALLOC_TABLE_FULL;
    int64_t need = live && st == 0 ? max(pages_for(L + n) - held, (int64_t)0) : 0;
    Pair ends{n, need};  // rows and pages up to and with this request
    Pair sums = block_scan(ends, sm.warp_sum, warps);
    const int64_t rows = sums.x, row_end = row0 + ends.x;
    if (row0 + rows > p.num_slots) {  // some request's rows do not fit: it asks for no page
      if (st == 0 && row_end > p.num_slots) st = MLA_KV_ALLOC_SLOTS_FULL;
      if (st != 0) need = 0;
      ends = Pair{0, need};
      sums = block_scan(ends, sm.warp_sum, warps);
    }
    const int64_t pages = sums.y, page_end = page0 + ends.y;
    if (need > 0 && page_end > count) st = MLA_KV_ALLOC_NO_PAGES;
    if constexpr (kFill) {
      sm.row_end[tid] = row_end;
      sm.first_page[tid] = page_end - need;
      sm.len[tid] = st == 0 ? L : -1;
      sm.held[tid] = held;
    }
    if (commit) {
      const bool grown = need > 0 && st == 0;
      if (live) {
        p.seq_lens_out[b] = st == 0 ? (int32_t)(L + n) : -1;
        p.held_out[b] = held + (grown ? (int32_t)need : 0);
        p.status[b] = st;
        p.cu[b + 1] = (int32_t)min(row_end, (int64_t)0x7fffffff);
      }
      // the requests that got pages come before those that got none: the sum only grows
      int64_t got = grown ? page_end : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) got = max(got, __shfl_xor_sync(0xffffffffu, got, o));
      if (lane == 0) sm.warp_sum[warp].x = got;
    }
    __syncthreads();
    if (commit)
      for (int w = 0; w < warps; ++w) taken = max(taken, sm.warp_sum[w].x);
    if constexpr (kFill) {
      const int nb = min(threads, p.batch - b0);
      const int64_t x_end = min(row0 + rows, hi);
      for (int64_t x0 = lo + (int64_t)warp * warp_rows; x0 < x_end; x0 += warps * warp_rows) {
        if (x0 + warp_rows <= row0) continue;  // (rows of an earlier chunk)
        int i = first_after(sm.row_end, nb, max(x0, row0));
        for (int k = 0; k < warp_rows; k += 32) {
          const int64_t x = x0 + k + lane;
          if (x < row0 || x >= x_end) continue;
          while (sm.row_end[i] <= x) ++i;
          int64_t slot = -1;
          const int len = sm.len[i], held_i = sm.held[i];
          if (len >= 0) {
            const int64_t pos = len + x - (i > 0 ? sm.row_end[i - 1] : row0);
            const int j = (int)(pos / kPageSize), off = (int)(pos % kPageSize);
            const int64_t at = (int64_t)(b0 + i) * p.max_pages + j;
            const bool fresh = j >= held_i;
            const int32_t page =
                fresh ? p.free_pages[count - 1 - sm.first_page[i] - (j - held_i)] : p.block_table[at];
            const bool in_cache = page >= 0 && page < p.num_pages;
            if (in_cache) slot = (int64_t)page * kPageSize + off;
            if (fresh && off == 0) {  // a page held before covers every cached token
              p.block_table[at] = page;
              if (p.page_tags != nullptr && in_cache) {
                const uint32_t tag = p.page_tags[page] + 1;
                p.page_tags[page] = tag;
                p.expected_tags[at] = tag;
              }
            }
          }
          p.slots[x] = (int32_t)slot;
        }
      }
    }
    row0 += rows;
    page0 += pages;
    __syncthreads();
  }
  if constexpr (kFill)
    for (int64_t x = max(row0, lo) + tid; x < hi; x += threads) p.slots[x] = -1;
  if (commit && tid == 0) {
    p.cu[0] = 0;
    p.free_count_out[0] = (int32_t)(count - taken);
  }
}

// Whether n int32 at a share memory with m int32 at b.
bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  if (sms <= 0) return MLA_ERR_CUDA;
  int64_t blocks = std::min<int64_t>((num_slots + kBlockRows - 1) / kBlockRows, sms);
  blocks = std::max<int64_t>(blocks, 1);
  // A warp bisects once per 128 rows, in a step of a few rows a request once per 32; one
  // block has the threads that its requests and rows keep busy.
  const int warp_rows = num_slots > kAllocThreads ? 128 : 32;
  const int64_t rows_per = ((num_slots + blocks - 1) / blocks + warp_rows - 1) / warp_rows * warp_rows;
  int threads = 128;
  while (threads < kAllocThreads && (blocks > 1 || threads < std::max<int64_t>(batch, num_slots)))
    threads *= 2;
  // Several blocks read the per-request inputs while block 0 writes its outputs: where
  // one of those shares memory with an input, they get a launch of their own.
  const void* ins[4] = {seq_lens, new_tokens, pages_held, free_count};
  const void* outs[5] = {seq_lens_out, pages_held_out, free_count_out, cu_tokens, request_status};
  bool apart = true;
  for (int i = 0; i < 4; ++i)
    for (int o = 0; o < 5; ++o)
      apart = apart && !overlap(ins[i], i == 3 ? 1 : batch, outs[o], o == 2 ? 1 : batch + (o == 3));
  if (blocks == 1 || apart) {
    kv_alloc_kernel<true, true><<<(unsigned)blocks, threads, 0, s>>>(p, rows_per, warp_rows);
  } else {
    kv_alloc_kernel<true, false><<<(unsigned)blocks, threads, 0, s>>>(p, rows_per, warp_rows);
    kv_alloc_kernel<false, true><<<1, threads, 0, s>>>(p, rows_per, warp_rows);
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
