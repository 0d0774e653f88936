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
// chunks of its size, and fills its own run of rows, a warp a run of them at a time: it
// finds their request by bisection in shared memory, and the row of a new page's first
// token also writes the page's table entry and tag. The page ids of new pages come from
// the free list itself, so that no row waits for another's table entry.
#include <algorithm>

#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kAllocThreads = 1024;    // at most; a step's few rows take fewer
constexpr int kAllocWarps = kAllocThreads / 32;
constexpr int64_t kBlockRows = 4096;   // rows that are worth a block of their own
// Rows that a warp fills at a time, with one search for their request: 32 in a step of few
// rows, 128 in larger calls, and 512 where the slot map has 4,096 entries a request (its size
// is what the host knows; a map that is much larger than its rows is taken for one of long
// requests): there most runs have one or two requests, and the warp looks their pages up at once. 32
// requests of 60k-140k new tokens take 10.3 us so (16.5 with 128 rows a time, each row its
// own lookup), 512 of 100-5,000 13.9 (12.3), 256 of four 15 (8.2); between 1,000 and 4,000
// rows a request the two are even.
constexpr int kFewRows = 32, kManyRows = 128, kPageRows = 512;
constexpr int64_t kRowsPerRequest = 4096;

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

// Running sums saturate at 2^31 - 1, past every row and page there can be: sums of
// non-negative numbers that saturate are still associative, and 32 bits suffice.
constexpr uint32_t kMost = 0x7fffffffu;
struct Pair {
  uint32_t x, y;
};
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
  return Pair{min(a.x + b.x, kMost), min(a.y + b.y, kMost)};
}
__device__ __forceinline__ Pair warp_scan(Pair v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair u{__shfl_up_sync(0xffffffffu, v.x, o), __shfl_up_sync(0xffffffffu, v.y, o)};
    if (lane >= o) v = plus(v, u);
  }
  return v;
}
// Inclusive running sums over the block's threads, in place; returns the totals.
__device__ __forceinline__ Pair block_scan(Pair& v, Pair* warp_sum, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  // every warp scans the warps' sums
  const Pair s = warp_scan(lane < warps ? warp_sum[lane] : Pair{0, 0}, lane);
  const int last = max(warp - 1, 0);
  const Pair before{__shfl_sync(0xffffffffu, s.x, last), __shfl_sync(0xffffffffu, s.y, last)};
  if (warp > 0) v = plus(v, before);
  const Pair total{__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31)};
  __syncthreads();  // the sums are no longer read
  return total;
}

// What the rows of a chunk's requests need.
struct AllocShared {
  Pair warp_sum[kAllocWarps];
  int32_t row_end[kAllocThreads];  // rows up to and with the request
  int32_t shift[kAllocThreads];    // token of row x = x + shift
  int32_t held[kAllocThreads];     // -1: refused
  int32_t fresh[kAllocThreads];    // page held + k = free_pages[fresh - k]
};

// First i < n with end[i] > x (n if there is none).
__device__ __forceinline__ int first_after(const int32_t* end, int n, int32_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int32_t pages_for(uint32_t tokens) {
  return (int32_t)(tokens / kPageSize + (tokens % kPageSize != 0));
}

// Rows x0 + [0, kPageRows) of the slot map, as far as they lie in begin .. end - 1, which belong to
// requests i and i + 1 of the chunk that starts at request b0. They lie in 11 pages at most:
// lane k looks up the k-th and enters it where it is new, and the rows take its id from there.
__device__ __forceinline__ void fill_by_page(const AllocParams& p, const AllocShared& sm, int b0, int i,
                                             int32_t x0, int32_t begin, int32_t end, int lane) {
  const int32_t cut = min(sm.row_end[i], end);  // where the second request's rows begin
  int32_t page = -1, shift[2] = {0, 0}, base[2] = {0, 0};  // lane of position x: x / 64 + base
  int64_t at = -1;  // block-table entry of a new page whose first token is here, else -1
  int lanes = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int32_t from = s ? cut : begin, to = s ? end : cut;
    if (from >= to) continue;
    const int32_t held = sm.held[i + s];
    shift[s] = held < 0 ? -from : sm.shift[i + s];
    const int32_t first = (from + shift[s]) / kPageSize;
    base[s] = lanes - first;
    const int32_t j = lane - base[s];
    if (held >= 0 && j >= first && j <= (to - 1 + shift[s]) / kPageSize) {
      const int64_t entry = (int64_t)(b0 + i + s) * p.max_pages + j;
      page = j < held ? p.block_table[entry] : p.free_pages[sm.fresh[i + s] - (j - held)];
      if (j >= held && j * kPageSize >= from + shift[s]) at = entry;
    }
    lanes += (to - 1 + shift[s]) / kPageSize - first + 1;
  }
  if (at >= 0) p.block_table[at] = page;
  if (page < 0 || page >= (int32_t)p.num_pages) page = -1;
  if (at >= 0 && page >= 0 && p.page_tags != nullptr) {
    const uint32_t tag = p.page_tags[page] + 1;
    p.page_tags[page] = tag;
    p.expected_tags[at] = tag;
  }
#pragma unroll
  for (int k = 0; k < kPageRows / 32; ++k) {
    const int32_t x = x0 + 32 * k + lane;
    const int s = x >= cut;
    const int32_t pos = (int32_t)((uint32_t)x + (uint32_t)(s ? shift[1] : shift[0]));
    const int32_t id = __shfl_sync(0xffffffffu, page, pos / kPageSize + (s ? base[1] : base[0]));
    if (x >= begin && x < end) p.slots[x] = id >= 0 ? id * kPageSize + pos % kPageSize : -1;
  }
}

// Rows x0 + [0, 32 * kRows) likewise, of requests i and on; a row looks its page up itself.
template <int kRows>
__device__ __forceinline__ void fill_by_row(const AllocParams& p, const AllocShared& sm, int b0, int i,
                                            int32_t x0, int32_t begin, int32_t end, int lane) {
  // all of a thread's page ids are asked for before the first is used, then all tags
  int32_t page[kRows], off[kRows];
  int64_t at[kRows];  // block-table entry of a new page's first token, else -1
  uint32_t tag[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int32_t x = x0 + 32 * k + lane;
    page[k] = -1;
    off[k] = 0;
    at[k] = -1;
    if (x < begin || x >= end) continue;
    while (sm.row_end[i] <= x) ++i;
    const int32_t held = sm.held[i];
    if (held < 0) continue;
    const int32_t pos = x + sm.shift[i], j = pos / kPageSize;
    const int64_t entry = (int64_t)(b0 + i) * p.max_pages + j;
    off[k] = pos % kPageSize;
    page[k] = j < held ? p.block_table[entry] : p.free_pages[sm.fresh[i] - (j - held)];
    // (a page held before covers every cached token: a new one starts at its token 0)
    if (j >= held && off[k] == 0) at[k] = entry;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const bool in_cache = page[k] >= 0 && page[k] < (int32_t)p.num_pages;
    if (at[k] >= 0) {
      p.block_table[at[k]] = page[k];
      if (p.page_tags == nullptr || !in_cache) at[k] = -1;
      else tag[k] = p.page_tags[page[k]] + 1;
    }
    const int32_t x = x0 + 32 * k + lane;
    if (x >= begin && x < end) p.slots[x] = in_cache ? page[k] * kPageSize + off[k] : -1;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    if (at[k] >= 0) {
      p.page_tags[page[k]] = tag[k];
      p.expected_tags[at[k]] = tag[k];
    }
}

// kRows > 0: rows [blockIdx.x * rows_per, + rows_per) of the slot map, kRows a warp at a
// time, with the new pages that begin there. kCommit: block 0 writes the per-request
// outputs, which may be the inputs: then no other block may still read them (one block in
// all, or a launch of its own).
template <int kRows, bool kCommit>
__global__ void __launch_bounds__(kAllocThreads)
    kv_alloc_kernel(const AllocParams p, const int64_t rows_per) {
  constexpr bool kFill = kRows > 0;
  __shared__ AllocShared sm;
  const int threads = blockDim.x, warps = threads >> 5;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool commit = kCommit && blockIdx.x == 0;
  const int32_t lo = (int32_t)min((int64_t)blockIdx.x * rows_per, p.num_slots);
  const int32_t hi = (int32_t)min((int64_t)lo + rows_per, p.num_slots);
  const int32_t count = min(max(p.free_count[0], 0), (int32_t)p.free_capacity);
  Pair done{0, 0};    // rows, and pages asked for, of the requests so far
  uint32_t taken = 0;  // pages taken so far
  for (int b0 = 0; b0 < p.batch; b0 += threads) {
    const int b = b0 + tid;
    const bool live = b < p.batch;
    const int32_t L = live ? p.seq_lens[b] : 0, held = live ? p.held[b] : 0;
    const int32_t asked = live ? p.new_tokens[b] : 0;
    const uint32_t n = (uint32_t)max(asked, 0);
    const int32_t fits = pages_for((uint32_t)L + n);
    uint32_t st = 0;
    if (L < 0 || asked < 0 || held < 0 || held > p.max_pages || pages_for((uint32_t)L) > held)
      st = MLA_KV_ALLOC_BAD_LENGTH;
    else if (fits > p.max_pages) st = MLA_KV_ALLOC_TABLE_FULL;
    uint32_t need = live && st == 0 ? (uint32_t)max(fits - held, 0) : 0u;
    Pair ends{n, need};  // rows and pages up to and with this request
    Pair sums = block_scan(ends, sm.warp_sum, warps);
    const Pair now = plus(done, sums);
    const uint32_t row_end = plus(done, ends).x, row_all = now.x;
    if (now.x > (uint32_t)p.num_slots) {  // some request's rows do not fit: it asks for no page
      if (st == 0 && row_end > (uint32_t)p.num_slots) st = MLA_KV_ALLOC_SLOTS_FULL;
      if (st != 0) need = 0;
      ends = Pair{0, need};
      sums = block_scan(ends, sm.warp_sum, warps);
    }
    const uint32_t page_end = plus(done, ends).y;
    if (need > 0 && page_end > (uint32_t)count) st = MLA_KV_ALLOC_NO_PAGES;
    if constexpr (kFill) {
      sm.row_end[tid] = (int32_t)row_end;
      sm.shift[tid] = (int32_t)((uint32_t)L - (row_end - n));
      sm.held[tid] = st == 0 ? held : -1;
      sm.fresh[tid] = (int32_t)((uint32_t)count - 1u - (page_end - need));
    }
    if (commit) {
      const bool grown = need > 0 && st == 0;
      if (live) {
        p.seq_lens_out[b] = st == 0 ? (int32_t)((uint32_t)L + n) : -1;
        p.held_out[b] = held + (grown ? (int32_t)need : 0);
        p.status[b] = st;
        p.cu[b + 1] = (int32_t)row_end;
      }
      // the requests that got pages come before those that got none: the sum only grows
      const uint32_t got = __reduce_max_sync(0xffffffffu, grown ? page_end : 0u);
      if (lane == 0) sm.warp_sum[warp].x = got;
    }
    __syncthreads();
    if (commit)
      taken = max(taken, __reduce_max_sync(0xffffffffu, lane < warps ? sm.warp_sum[lane].x : 0u));
    if constexpr (kFill) {
      const int nb = min(threads, p.batch - b0);
      const int32_t from = (int32_t)done.x, to = min((int32_t)row_all, hi);
      for (int32_t x0 = lo + warp * kRows; x0 < to; x0 += warps * kRows) {
        if (x0 + kRows <= from) continue;  // (rows of an earlier chunk)
        const int32_t begin = max(x0, from), end = min(x0 + kRows, to);
        // None of these rows is this chunk's: it has no rows here (none at all, or the rows
        // before it end beyond the slot map), and no request of it would be found.
        if (begin >= end) continue;
        const int i = first_after(sm.row_end, nb, begin);
        if constexpr (kRows == kPageRows) {
          if (i + 2 >= nb || sm.row_end[i + 1] >= end) {
            fill_by_page(p, sm, b0, i, x0, begin, end, lane);
          } else {
            for (int32_t x = x0; x < end; x += kManyRows)
              if (x + kManyRows > begin)
                fill_by_row<kManyRows / 32>(p, sm, b0, x <= begin ? i : first_after(sm.row_end, nb, x), x,
                                            begin, end, lane);
          }
        } else {
          fill_by_row<kRows / 32>(p, sm, b0, i, x0, begin, end, lane);
        }
      }
    }
    done = Pair{row_all, plus(done, sums).y};
    __syncthreads();
  }
  if constexpr (kFill)
    for (int32_t x = max((int32_t)done.x, lo) + tid; x < hi; x += threads) p.slots[x] = -1;
  if (commit && tid == 0) {
    p.cu[0] = 0;
    p.free_count_out[0] = count - (int32_t)taken;
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
  if (num_pages > 0x7fffffff / kPageSize || num_slots > 0x7fff0000LL ||
      free_capacity > 0x7fff0000LL ||  // (sums and runs of rows end below 2^31)
      max_pages > 0x7fffffff / kPageSize)
    return MLA_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !cu_tokens) return MLA_ERR_INVALID_ARG;
  if (batch > 0 && (!seq_lens || !new_tokens || !pages_held || !block_table || !seq_lens_out ||
                    !pages_held_out || !request_status))
    return MLA_ERR_INVALID_ARG;
  if ((free_capacity > 0 && !free_pages) || (num_slots > 0 && !slot_mapping))
    return MLA_ERR_INVALID_ARG;
  // (an array without an entry may have no address)
  if (batch > 0 && num_pages > 0 && (page_tags == nullptr) != (expected_tags == nullptr))
    return MLA_ERR_INVALID_ARG;
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
  const int warp_rows = num_slots <= kAllocThreads ? kFewRows
                        : num_slots >= kRowsPerRequest * batch ? kPageRows
                                                               : kManyRows;
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
  const bool at_once = blocks == 1 || apart;
  const auto fill =
      warp_rows == kFewRows ? kv_alloc_kernel<kFewRows, true>
      : warp_rows == kManyRows
          ? (at_once ? kv_alloc_kernel<kManyRows, true> : kv_alloc_kernel<kManyRows, false>)
          : (at_once ? kv_alloc_kernel<kPageRows, true> : kv_alloc_kernel<kPageRows, false>);
  fill<<<(unsigned)blocks, threads, 0, s>>>(p, rows_per);
  if (!at_once) kv_alloc_kernel<0, true><<<1, threads, 0, s>>>(p, rows_per);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
