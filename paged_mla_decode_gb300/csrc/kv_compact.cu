// kv_compact.cu -- move the kept nodes' cache entries together after a tree's verification.
//
// "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
// custom speculative decoding ...": drafted tokens are verified in parallel, so the cache
// holds an entry of every node of a tree, in node order, and a verification that keeps
// nodes path[1], path[2], ... leaves gaps between theirs. The entries move as they are
// stored (no value is converted), in every layer's pages.
//
// A few KB a request and layer move, behind a chain of dependent reads (how many were kept,
// which, their pages): latency bounds a call. So a block resolves its request's moves once,
// with a thread each, and applies them to several layers. All of an entry's 16-byte columns
// of a pass are in registers before any is written, so an entry may be read and overwritten.
// 32 requests' trees of 16 nodes in 61 layers' e4m3 pages 5.5 us, 16 of 32 nodes in a 4-bit
// cache 5.3.
#include <algorithm>

#include "kv_e2m1.cuh"
#include "mla_common.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;  // 16-byte columns of a thread in a pass
constexpr int kMaxMoves = MLA_MAX_TREE_NODES - 1;
constexpr int kExpBytes = kDEntry / kE2m1Block / 2;  // 9 bytes of exponents of a 4-bit entry

struct CompactParams {
  uint8_t* kv;
  int layers, layers_a_block;
  int64_t layer_stride;  // bytes
  int64_t num_pages;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* path;
  const int32_t* accepted;
  int max_nodes;
  int entry_bytes;  // of a row of [64][entry] pages; 4-bit: see below
};

// One 16-byte column of an entry; a 4-bit entry's last one is its nine exponent bytes.
template <bool kE2m1>
struct Column {
  static __device__ __forceinline__ uint4 load(const uint8_t* page, int t, int c, int entry) {
    if constexpr (!kE2m1) return *reinterpret_cast<const uint4*>(page + (int64_t)t * entry + 16 * c);
    if (c < kDEntry / kE2m1Block)
      return *reinterpret_cast<const uint4*>(page + (c * kPageSize + t) * 16);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kExpBytes; ++i)
      w[i / 4] |= (uint32_t)page[e2m1_exp_offset(2 * i, t)] << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void store(uint8_t* page, int t, int c, int entry, const uint4& v) {
    if constexpr (!kE2m1) {
      *reinterpret_cast<uint4*>(page + (int64_t)t * entry + 16 * c) = v;
      return;
    }
    if (c < kDEntry / kE2m1Block) {
      *reinterpret_cast<uint4*>(page + (c * kPageSize + t) * 16) = v;
      return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kExpBytes; ++i)
      page[e2m1_exp_offset(2 * i, t)] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
};

template <bool kE2m1>
__global__ void __launch_bounds__(kThreads) kv_compact_kernel(const CompactParams p) {
  __shared__ int64_t s_from[kMaxMoves], s_to[kMaxMoves];  // slots
  __shared__ int s_count;
  const int b = blockIdx.x, tid = threadIdx.x;
  griddep_wait();  // all earlier work in the stream is complete
  griddep_launch_dependents();
  if (tid == 0) s_count = 0;
  const int a = p.accepted[b], L = p.seq_lens[b];
  if (a < 1 || a >= p.max_nodes || L < a + 1 || (int64_t)L > (int64_t)p.max_pages * kPageSize) return;
  const int base = L - a - 1;
  __syncthreads();
  if (tid < 64) {  // move `tid`: node path[tid + 1] to place tid + 1
    int64_t from = -1, to = -1;
    if (tid < a) {
      const int node = p.path[(int64_t)b * p.max_nodes + tid + 1];
      const int src = base + node, dst = base + tid + 1;
      if (node >= 0 && node < p.max_nodes && node != tid + 1 && src < p.max_pages * (int64_t)kPageSize) {
        const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
        const int ps = table[src / kPageSize], pd = table[dst / kPageSize];
        if (ps >= 0 && ps < p.num_pages && pd >= 0 && pd < p.num_pages) {
          from = (int64_t)ps * kPageSize + src % kPageSize;
          to = (int64_t)pd * kPageSize + dst % kPageSize;
        }
      }
    }
    const unsigned have = __ballot_sync(0xffffffffu, from >= 0);
    int at = 0;
    if ((tid & 31) == 0) at = atomicAdd(&s_count, __popc(have));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(have & ((1u << (tid & 31)) - 1));
    if (from >= 0) {
      s_from[at] = from;
      s_to[at] = to;
    }
  }
  __syncthreads();
  const int moves = s_count;
  if (moves == 0) return;
  const int columns = kE2m1 ? kDEntry / kE2m1Block + 1 : p.entry_bytes / 16;
  const int first = blockIdx.y * p.layers_a_block;
  const int layers = min(p.layers_a_block, p.layers - first);
  const int64_t page_bytes = kE2m1 ? kE2m1PageBytes : (int64_t)kPageSize * p.entry_bytes;
  // items are (layer, column) times moves; a pass takes whole columns of whole layers' entries
  const int per_pass = kThreads * kLoads / moves, groups = layers * columns;
  for (int g0 = 0; g0 < groups; g0 += per_pass) {
    const int items = min(per_pass, groups - g0) * moves;
    uint4 v[kLoads];
    auto item = [&](int u, const int64_t* slots, int& t, int& c) -> uint8_t* {
      const int i = u * kThreads + tid;
      // neighbouring threads take neighbouring columns of one move
      const int per = items / moves, m = i / per, g = g0 + (i - m * per);
      const int layer = g / columns;
      c = g - layer * columns;
      const int64_t slot = slots[m];
      t = (int)(slot % kPageSize);
      return p.kv + (first + layer) * p.layer_stride + slot / kPageSize * page_bytes;
    };
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (u * kThreads + tid < items) {
        int t, c;
        const uint8_t* page = item(u, s_from, t, c);
        v[u] = Column<kE2m1>::load(page, t, c, p.entry_bytes);
      }
    }
    __syncthreads();  // a column's entries are all read before one of them is written
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (u * kThreads + tid < items) {
        int t, c;
        uint8_t* page = item(u, s_to, t, c);
        Column<kE2m1>::store(page, t, c, p.entry_bytes, v[u]);
      }
    }
  }
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_kv_compact(void* kv_pages, int num_layers, int64_t layer_stride,
                                     int64_t num_pages, int page_size, int kv_dtype,
                                     const int32_t* block_table, int max_pages,
                                     const int32_t* seq_lens, const int32_t* path,
                                     const int32_t* num_accepted, int batch, int max_nodes,
                                     mla_stream_t stream) {
  using namespace mla;
  if (batch < 0 || num_layers < 0 || num_pages < 0 || max_pages < 1 || max_nodes < 1 ||
      max_nodes > MLA_MAX_TREE_NODES)
    return MLA_ERR_INVALID_ARG;
  if (page_size != kPageSize) return MLA_ERR_UNSUPPORTED;
  if (kv_dtype != MLA_KV_E4M3 && kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_E2M1)
    return MLA_ERR_INVALID_ARG;
  const int entry = kv_dtype == MLA_KV_BF16 ? 2 * kDEntry : kDEntry;
  const int64_t page_bytes = kv_dtype == MLA_KV_E2M1 ? kE2m1PageBytes : (int64_t)kPageSize * entry;
  if (num_layers > 1 && (layer_stride < num_pages * page_bytes || layer_stride % 16 != 0))
    return MLA_ERR_INVALID_ARG;
  if (num_pages > (int64_t)(0x7fffffff / kPageSize) || (int64_t)batch * max_pages > 0x7fffffffLL ||
      max_pages > 0x7fffffff / kPageSize || num_layers > 65535)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0 || num_layers == 0) return MLA_OK;
  if (!kv_pages || !block_table || !seq_lens || !path || !num_accepted) return MLA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(kv_pages) & 15u) return MLA_ERR_INVALID_ARG;
  const void* ptrs[4] = {block_table, seq_lens, path, num_accepted};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MLA_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MLA_ERR_CUDA;
  CompactParams p;
  p.kv = static_cast<uint8_t*>(kv_pages);
  p.layers = num_layers;
  // about four blocks an SM
  p.layers_a_block = (int)std::max<int64_t>(1, (int64_t)batch * num_layers / (4 * sms));
  p.layer_stride = layer_stride;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.path = path;
  p.accepted = num_accepted;
  p.max_nodes = max_nodes;
  p.entry_bytes = entry;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch, (unsigned)((num_layers + p.layers_a_block - 1) / p.layers_a_block));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, kv_dtype == MLA_KV_E2M1 ? kv_compact_kernel<true> : kv_compact_kernel<false>, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
