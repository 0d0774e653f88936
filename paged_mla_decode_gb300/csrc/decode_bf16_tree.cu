// decode_bf16_tree.cu -- split-KV tree decode over a bfloat16 cache (mla_decode_tree).
//
// A CTA walks its run of (row tile, page) steps (TreePlan), one 64-token page per step:
//   S [64 rows x 64 tokens]   = Q . page^T            (M = 64, 36 steps of 16 dims)
//   O^T[512 x 64 rows]       += V^T . P^T             V = the page's first 512 dims
// with the page's bytes as tcgen05.mma kind::f16 operands as they are stored: TMA brings a page
// as nine 128-byte-swizzled chunks of 64 dims, which are K as they lie and V through an
// MN-major descriptor (no distinct values: "How to serve trillions of tokens ...", section
// "First, understand the workload"). All query rows of a request attend over the one latent
// head ("vLLM x AgentX", section "Kimi K3").
//
// A page is 73,728 bytes and the tile's query as many, so two pages fit beside it, and P
// (bf16, 8 KB) takes the place of its own page's rotary chunk, which QK has read by then.
// That bounds it: copy, QK, softmax and PV of a page follow each other in its slot. 16 sessions
// of 32k-140k tokens, 12 nodes of 64 heads: a call of 3,248 us, 1.8 us a page and SM, 756
// TFLOP/s; 32 requests of up to 4k, 31 nodes of 32 heads: 300 us, 477. So QK starts on the first
// third of a page (1% of such 32 requests, when the issue of MMAs took longer), a third of the next
// page comes as soon as PV has passed the one in its place (6% of the 16 sessions; five groups
// instead of three cost them 50%), and L2 is asked for pages four ahead.
// P = 2^(s - m) with m a running maximum that rises when a page's lies more than 2^7 above it:
// bf16 has float's range, so P of a page far below m keeps its 8 bits (each rounded once,
// 2^-8 of itself at most; the normaliser sums the exact P).
//
// Warp roles (352 threads):
//   warps 0-7  softmax and epilogue: row h of S is TMEM lane 32*(h/16) + h%16 (M = 64); thread
//              (w, lane) handles row 16*(w%4) + lane%16 and the 16 tokens 32*(w/4) +
//              16*(lane/16) .. +15 of a page. For O^T, lane t is dim t of each 128-dim block.
//   warp 8     TMA producer (lane 0): page ids from the block table a window ahead, the query
//              tile at a piece's start, pages into the two slots; warps 9, 10 issue QK and PV;
//              warp 9 allocates TMEM.
// TMEM (512 columns): S buffers [0,64) [64,128), O^T [256,512).
//
// Every wait is bounded (2 s); on timeout the CTA records MLA_DEVICE_ERR_TIMEOUT, stops, drains
// its MMAs and copies (bounded, 2 s) and frees TMEM; tests/test_gpu_tree_bf16_timeout.py runs that.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "page_walk.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kSmWarps = 8, kSmThreads = 32 * kSmWarps;
constexpr int kTmaWarp = 8, kQkWarp = 9;  // (10: PV)
constexpr int kThreads = 32 * 11;
constexpr int kTileRows = 64;
constexpr int kChunks = kDEntry / 64;               // 9 chunks of 64 dims
constexpr int kChunkBytes = kPageSize * 128;        // 8192
constexpr int kPageBytes = kChunks * kChunkBytes;   // 73,728
constexpr int kSlots = 2;
constexpr int kGroups = 3;                          // QK starts on a third of a page
constexpr int kPrefetch = 4;                        // pages ahead that L2 is asked for
constexpr float kRescaleThresh = 7.0f;              // log2 units
// Limits of a wait on another role, which a test build lowers to make the timeout path run, and of
// a wait for copies and MMAs already issued.
#ifndef MLA_PIPELINE_WAIT_NS
#define MLA_PIPELINE_WAIT_NS 2000000000ull
#endif
constexpr uint64_t kWaitNs = MLA_PIPELINE_WAIT_NS;
constexpr uint64_t kDrainWaitNs = 2000000000ull;
constexpr int kDescRing = 64;    // page descriptors in flight
constexpr int kTableAhead = 32;  // pages described (block-table read started) before issue

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t s_col(uint32_t b) { return 64u * b; }
constexpr uint32_t kOCol = 256;

constexpr int kOffQ = kSlots * kPageBytes;
constexpr int kOffAlpha = kOffQ + kPageBytes;            // float [64]
constexpr int kOffLinv = kOffAlpha + 256;                // float [64]
constexpr int kOffPmax = kOffLinv + 256;                 // float [2 pages][2 halves][64]
constexpr int kOffLsum = kOffPmax + 1024;                // float [2 halves][64]
constexpr int kOffFlags = kOffLsum + 512;                // int [4]
constexpr int kOffPlan = kOffFlags + 16;                 // int64 [6]
constexpr int kOffDesc = kOffPlan + 48;                  // PageDesc [kDescRing]
constexpr int kOffBar = kOffDesc + 16 * kDescRing;
enum Bar {
  BAR_PAGE_FULL = 0,                  // [2][3] three of the page's chunks landed (or there are none)
  BAR_PV_DONE = BAR_PAGE_FULL + 2 * kGroups,    // [2] PV of the page in the slot: slot, P and O^T free
  BAR_S_FULL = BAR_PV_DONE + 2,       // [2] page j: buffer j % 2
  BAR_S_EMPTY = BAR_S_FULL + 2,       // [2] (softmax warps)
  BAR_P_FULL = BAR_S_EMPTY + 2,       // [2] (softmax warps)
  BAR_O_FULL = BAR_P_FULL + 2,
  BAR_O_EMPTY = BAR_O_FULL + 1,       // (softmax warps)
  BAR_Q_FULL = BAR_O_EMPTY + 1,       // the query tile's bytes landed
  BAR_Q_EMPTY = BAR_Q_FULL + 1,       // QK of the piece's last page is done
  BAR_DRAIN = BAR_Q_EMPTY + 1,        // [2] one per issuer warp
  // [2][kGroups] the page's PV has read the third in the slot
  BAR_FREE = BAR_DRAIN + 2,
#ifdef MLA_TEST_STALL_QK
  // Test build only: a barrier that nothing ever completes, on which the QK issuer waits before its
  // third page (as in decode_fp8.cu).
  BAR_TEST_STALL = BAR_FREE + 2 * kGroups,
  kNumBars
#else
  kNumBars = BAR_FREE + 2 * kGroups
#endif
};
constexpr int kOffTmem = kOffBar + 8 * kNumBars;
constexpr int kSmemBytes = kOffTmem + 16 + 1024;  // slack for the 1024 alignment
static_assert(kSmemBytes <= 227 * 1024, "shared memory map exceeds 227 KB");

enum Flag { F_ABORT = 0, F_PIECE_BAD = 1 };

struct Bf16TreeParams {
  const uint8_t* kv;
  int64_t num_pages;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seq_lens;
  int batch, tiles, tile_rows;
  float score_mul;  // sm_scale * log2(e) * kv_scale
  float kv_scale;
  int G;
  DecodeWorkspace ws;
  const uint64_t* tree_mask;
  const int32_t* num_nodes;
  int max_nodes, node_heads;
  int query_rows;  // of a request
};

__device__ __forceinline__ void bar_softmax() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(kSmThreads) : "memory");
}
__device__ __forceinline__ bool bar_softmax_or(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)pred), "n"(kSmThreads)
      : "memory");
  return r != 0;
}
// Two floats as bf16, the first lowest.
__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__global__ void __launch_bounds__(kThreads, 1)
    decode_bf16_tree_kernel(const Bf16TreeParams p, const __grid_constant__ CUtensorMap kv_map,
                            const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_a = smem_u32(smem_raw);
  const uint32_t sbase = (raw_a + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_a);
  float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);
  float* linv_s = reinterpret_cast<float*>(smem + kOffLinv);
  float* pmax_s = reinterpret_cast<float*>(smem + kOffPmax);
  float* lsum_s = reinterpret_cast<float*>(smem + kOffLsum);
  volatile int* flags = reinterpret_cast<volatile int*>(smem + kOffFlags);
  int64_t* s_plan = reinterpret_cast<int64_t*>(smem + kOffPlan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmem);
  auto bar = [&](int i) -> uint32_t { return sbase + kOffBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the compiler sees that it is a warp's)
  const int c = blockIdx.x;
  griddep_wait();  // all earlier work in the stream is complete
  TreePlan plan{p.seq_lens, p.num_nodes, p.batch, p.max_nodes, p.node_heads, p.tiles, p.tile_rows,
                p.max_pages, kPageSize, p.G, 0};
  if (warp == 0) {
    TreePlan pl = plan;
    pl.set_total(plan_total_tiles_warp(pl));
    const int64_t xb = c < pl.G ? pl.cta_start(c) : 0;
    const RowCursor f = plan_find_row_warp(pl, xb, c == 0, p.ws.row_base, p.ws.row_np, p.ws.status);
    if (lane == 0) {
      s_plan[0] = pl.T;
      s_plan[1] = f.r;
      s_plan[2] = f.rt;
      s_plan[3] = f.t;
      s_plan[4] = f.base;
      s_plan[5] = f.n;
    }
  }
  if (warp == kTmaWarp && lane == 0) {
    tc::prefetch_tensormap(&kv_map);
    tc::prefetch_tensormap(&q_map);
    for (int i = 0; i < kNumBars; ++i) {
      const bool by_softmax = (i >= BAR_S_EMPTY && i < BAR_P_FULL + 2) || i == BAR_O_EMPTY;
      tc::mbar_init(bar(i), by_softmax ? kSmWarps : 1);
    }
    tc::fence_mbar_init();
    flags[F_ABORT] = 0;
    flags[F_PIECE_BAD] = 0;
  }
  if (warp == kQkWarp) {
    tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tc::tmem_relinquish();
  }
  // rows that TMA does not write (a request of fewer than 64) are zeros
  if (p.tile_rows < kTileRows) {
    const int units = (kTileRows - p.tile_rows) * 8;  // 16-byte pieces of a chunk
    for (int i = tid; i < kChunks * units; i += kThreads) {
      const int ch = i / units, u = i - ch * units;
      asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                       sbase + kOffQ + ch * kChunkBytes + p.tile_rows * 128 + u * 16),
                   "r"(0u));
    }
    tc::fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();  // the merge may be scheduled (it waits for this grid)
  plan.set_total(s_plan[0]);
  const bool works = c < plan.G;
  const int64_t x_begin = works ? plan.cta_start(c) : 0, x_end = works ? plan.cta_start(c + 1) : 0;
  const uint32_t tmem = *tmem_slot;
  const RowCursor cur0{(int)s_plan[1], s_plan[2], (int)s_plan[3], (int)s_plan[4], (int)s_plan[5]};
  const int H = p.tile_rows;
  auto abort_cta = [&]() {
    flags[F_ABORT] = 1;
    atomicOr(p.ws.status, MLA_DEVICE_ERR_TIMEOUT);
  };
  const int64_t npages = x_end - x_begin;
  const PageDesc* desc = reinterpret_cast<const PageDesc*>(smem + kOffDesc);
  if (x_begin < x_end) {
    if (warp == kTmaWarp) {
      // =================== TMA producer (lane 0) ===================
      if (lane == 0) {
        const uint64_t pol = l2_evict_first_policy();
        PageDesc* ring = reinterpret_cast<PageDesc*>(smem + kOffDesc);
        PageWalker<TreePlan> pw;
        pw.init(plan, cur0, c, x_begin, x_end);
        int64_t jn = 0;  // next page to describe
        auto describe_next = [&]() {
          PageDesc& d = ring[jn % kDescRing];
          d.valid = (int8_t)pw.valid_tokens();
          const int before = pw.cur.n - plan.nodes(pw.cur.r / plan.tiles);
          d.context = (int8_t)min(before - pw.page_in_row() * kPageSize, kPageSize);
          d.flags = (int16_t)((pw.piece_start() ? kDescPieceStart : 0) |
                              (pw.piece_end() ? kDescPieceEnd : 0));
          d.row = pw.qrow;
          d.slot = pw.slot;
          cp_async_4(smem_u32(&d.page), p.block_table + pw.bt_row + pw.page_in_row());
          cp_async_commit();
          pw.next();
          ++jn;
        };
        // (pages whose ids are waited for at page j: it and those that L2 is asked for)
        while (jn <= kPrefetch && jn < npages) describe_next();
        int64_t j = 0, asked = 0;
        int piece = 0, part = 0;  // thirds of page j that are on their way
        bool ok = true;
        for (; j < npages; ++j) {
          cp_async_wait_upto<kTableAhead>((int)max(jn - j - 1 - kPrefetch, (int64_t)0));
          PageDesc* d = ring + j % kDescRing;
          for (; asked < jn && asked <= j + kPrefetch; ++asked) {
            const int32_t ahead = ring[asked % kDescRing].page;
            if (asked >= j + kSlots && ahead >= 0 && (int64_t)ahead < p.num_pages)
              tc::prefetch_l2_bulk(p.kv + (int64_t)ahead * kPageBytes, (uint32_t)kPageBytes);
          }
          const bool page_ok = d->page >= 0 && (int64_t)d->page < p.num_pages;
          if (page_ok) d->flags |= kDescPageOk;
          if (d->flags & kDescPieceStart) {
            // the piece's query rows (a last tile may reach into the next request, or past the
            // end: zeros; no such row is live)
            if (piece > 0 && (!tc::mbar_wait(bar(BAR_Q_EMPTY), (uint32_t)(piece - 1) & 1, kWaitNs) ||
                              flags[F_ABORT])) {
              ok = false;
              break;
            }
            ++piece;
            const int b = d->row / p.tiles;
            const int y = b * p.query_rows + (d->row - b * p.tiles) * H;
            tc::mbar_arrive_expect_tx(bar(BAR_Q_FULL), (uint32_t)(kChunks * H * 128));
            for (int ch = 0; ch < kChunks; ++ch)
              tc::tma_load_2d(sbase + kOffQ + ch * kChunkBytes, &q_map, 64 * ch, y, bar(BAR_Q_FULL));
          }
          const int slot = (int)(j % kSlots);
          for (int g = 0; g < kGroups && ok; ++g) {  // a third at a time, as it becomes free
            const uint32_t full = bar(BAR_PAGE_FULL + kGroups * slot + g);
            if (j >= kSlots && (!tc::mbar_wait(bar(BAR_FREE + kGroups * slot + g), (uint32_t)(j / kSlots - 1) & 1, kWaitNs) ||
                                flags[F_ABORT])) {
              ok = false;
              break;
            }
            ++part;
            if (!page_ok) {  // no copy; every token of the page is masked, its value rows zeroed
              tc::mbar_arrive(full);
              continue;
            }
            tc::mbar_arrive_expect_tx(full, (uint32_t)(kPageBytes / kGroups));
            const uint32_t to = sbase + slot * kPageBytes;
            const int y = d->page * kPageSize;
            for (int ch = 3 * g; ch < 3 * g + 3; ++ch)
              tc::tma_load_2d_hint(to + ch * kChunkBytes, &kv_map, 64 * ch, y, full, pol);
          }
          if (!ok) break;
          part = 0;
          for (int u = 0; u < 2 && jn < npages && jn <= j + kTableAhead; ++u) describe_next();
        }
        cp_async_wait<0>();
        if (!ok) abort_cta();
        // no copy may land after the CTA exits: wait for the last issued pages and query (a wait
        // that runs out has been long enough for all)
        bool landed = true;
        for (int64_t jj = j > kSlots ? j - kSlots : 0; jj < j; ++jj)
          for (int g = 0; g < kGroups; ++g)
            landed = landed && tc::mbar_wait(bar(BAR_PAGE_FULL + kGroups * (int)(jj % kSlots) + g),
                                             (uint32_t)(jj / kSlots) & 1, kDrainWaitNs);
        for (int g = 0; g < part; ++g)
          landed = landed && tc::mbar_wait(bar(BAR_PAGE_FULL + kGroups * (int)(j % kSlots) + g),
                                           (uint32_t)(j / kSlots) & 1, kDrainWaitNs);
        if (piece > 0) tc::mbar_wait(bar(BAR_Q_FULL), (uint32_t)(piece - 1) & 1, kDrainWaitNs);
      }
      __syncwarp();
    } else if (warp >= kQkWarp) {
      // =================== MMA issuers (two warps) ===================
      // The whole warp runs the loop, with values that the compiler knows to be a warp's (an MMA
      // takes its operands from uniform registers), and one elected thread issues the MMAs: a
      // loop of lane 0 alone took 70 cycles for each.
      constexpr uint32_t id_qk = tc::idesc_f16(64, 64, true, false, false);
      constexpr uint32_t id_pv = tc::idesc_f16(128, 64, true, true, false);  // A = V^T, MN-major
      const bool is_qk = warp == kQkWarp;
      auto wait = [&](int b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar(b), parity, kWaitNs));
      };
      int piece = 0, left = 0, in_piece = 0;  // pages of the piece
      bool ok = true;
      PageWalker<TreePlan> pw;  // piece boundaries
      pw.init(plan, cur0, c, x_begin, x_end);
      const uint64_t qa = tc::smem_desc_sw128(sbase + kOffQ, 16, 1024);
      const uint32_t pages = __shfl_sync(0xffffffffu, (uint32_t)npages, 0);
      for (uint32_t k = 0; k < pages && ok; ++k) {
        if (__any_sync(0xffffffffu, flags[F_ABORT])) {
          ok = false;
          break;
        }
        const uint32_t slot = k % kSlots, par = (k / kSlots) & 1;
        const uint32_t page = sbase + slot * kPageBytes;
        if (left == 0) {
          left = in_piece = __shfl_sync(0xffffffffu, pw.piece_pages(), 0);
          ok = wait(is_qk ? BAR_Q_FULL : BAR_O_EMPTY, (uint32_t)piece & 1);
          ++piece;
        }
        if (is_qk) {
#ifdef MLA_TEST_STALL_QK
          if (k == 2) ok = ok && wait(BAR_TEST_STALL, 0);
#endif
          if (ok && k >= 2) ok = wait(BAR_S_EMPTY + slot, ((k >> 1) - 1) & 1);
          const uint64_t kb = tc::smem_desc_sw128(page, 16, 1024);
          const uint32_t d_s = tmem + s_col(k & 1u);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            if (ok) ok = wait(BAR_PAGE_FULL + kGroups * slot + g, par);
            if (!ok) break;
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
              for (int s = 4 * kChunks / kGroups * g; s < 4 * kChunks / kGroups * (g + 1); ++s) {
                const uint32_t at = (s >> 2) * kChunkBytes + (s & 3) * 32;
                tc::mma_f16_ss(d_s, tc::desc_at(qa, at), tc::desc_at(kb, at), id_qk, s > 0);
              }
            }
          }
          if (!ok) break;
          if (tc::elect_one()) {
            tc::mma_commit(bar(BAR_S_FULL + (int)(k & 1)));
            if (left == 1) tc::mma_commit(bar(BAR_Q_EMPTY));
          }
        } else {
          if (ok) ok = wait(BAR_P_FULL + slot, par);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t va = tc::smem_desc_sw128(page, kChunkBytes, 1024);
          const uint64_t pb = tc::smem_desc_sw128(page + (kChunks - 1) * kChunkBytes, 16, 1024);
          if (tc::elect_one()) {
#pragma unroll
            for (int blk = 0; blk < 4; ++blk) {  // (two chunks a block: chunks 3g .. 3g + 2 are read by g + 2 of them)
#pragma unroll
              for (int s = 0; s < 4; ++s)
                tc::mma_f16_ss(tmem + kOCol + 64 * blk, tc::desc_at(va, 2 * blk * kChunkBytes + s * 2048),
                               tc::desc_at(pb, 32 * s), id_pv, 1);
              if (blk > 0) tc::mma_commit(bar(BAR_FREE + kGroups * slot + blk - 1));
            }
            tc::mma_commit(bar(BAR_PV_DONE + slot));
            if (left == 1) tc::mma_commit(bar(BAR_O_FULL));
          }
        }
        if (--left == 0) {
          pw.to_piece_end(in_piece);
          pw.next();
        }
      }
      if (!ok && lane == 0) abort_cta();
      // drain: every MMA this warp issued has finished before TMEM is freed
      const int db = BAR_DRAIN + (is_qk ? 0 : 1);
      if (tc::elect_one()) tc::mma_commit(bar(db));
      if (!tc::mbar_wait(bar(db), 0, kDrainWaitNs)) atomicOr(p.ws.status, MLA_DEVICE_ERR_TIMEOUT);
      __syncwarp();
    } else {
      // =================== softmax + epilogue (warps 0-7) ===================
      const int q4 = warp & 3, g = warp >> 2;
      const int h = 16 * q4 + (lane & 15);
      const int c16 = 2 * g + (lane >> 4);  // this thread's 16-token chunk of a page
      const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
      float m = -INFINITY, lpart = 0.f;
      uint64_t nodes_seen = 0;
      bool row_live = false, ok = true;
      int piece = 0;
      auto zero_o = [&]() {  // O^T (PV always accumulates); this warp's lanes, rows 32g ..
        uint32_t zz[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zz[i] = 0u;
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) tc::tmem_st32(tmem + lane_base + kOCol + 64 * blk + 32 * g, zz);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(BAR_O_EMPTY));
      };
      zero_o();
      const uint32_t pages = (uint32_t)npages;
      for (uint32_t j = 0; j < pages; ++j) {
        const uint32_t slot = j % kSlots, par = (j / kSlots) & 1;
        const uint32_t page_base = sbase + slot * kPageBytes;
        // (a failed wait, like a stop by another role, is acted on at the block barrier below)
        bool stop = flags[F_ABORT] != 0;
        // (S_FULL: all of the page has landed; the chunks' barriers make it visible here too)
        if (!tc::mbar_wait(bar(BAR_S_FULL + slot), par, kWaitNs)) {
          flags[F_ABORT] = 1;
          stop = true;
        }
#pragma unroll
        for (int third = 0; third < kGroups; ++third)
          if (!tc::mbar_wait(bar(BAR_PAGE_FULL + kGroups * slot + third), par, kWaitNs)) {
            flags[F_ABORT] = 1;
            stop = true;
          }
        const PageDesc d = desc[j % kDescRing];
        const bool ps = d.flags & kDescPieceStart, pe = d.flags & kDescPieceEnd;
        const bool page_ok = d.flags & kDescPageOk;
        const int nvis = page_ok ? d.valid : 0;
        const bool has_nodes = d.context < kPageSize && page_ok;
        if (tid == 0 && !page_ok && !stop) {
          flags[F_PIECE_BAD] = 1;
          atomicOr(p.ws.status, MLA_DEVICE_ERR_BAD_PAGE);
        }
        if (ps && !stop) {
          nodes_seen = h < H ? tree_row_mask(plan, p.tree_mask, d.row, h) : 0;
          row_live = h < H && tree_row_live(plan, d.row, h);
          m = -INFINITY;
          lpart = 0.f;
        }
        tc::fence_after_sync();
        uint32_t sr[16];
        tc::tmem_ld16x2_16(tmem + lane_base + s_col(j & 1u) + 32u * (uint32_t)g, sr);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(BAR_S_EMPTY + slot));
        float s[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 v = mul2(make_float2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])),
                                make_float2(p.score_mul, p.score_mul));
          s[i] = v.x;
          s[i + 1] = v.y;
        }
        if (has_nodes) {
          // (the nodes are a request's last tokens: a page with any of them, or with fewer than
          // 64 tokens, has this test; a node behind the request's last is in no mask)
          const uint32_t seen = tree_visible(nodes_seen, d.context, 16 * c16);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!((seen >> i) & 1u)) s[i] = -INFINITY;
        } else if (nvis < kPageSize) {  // a bad page id
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = -INFINITY;
        }
        float tm = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) tm = fmaxf(tm, s[i]);
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 16));
        if (lane < 16) pmax_s[(j & 1) * 128 + g * 64 + h] = tm;
        const bool any = bar_softmax_or((!ps && tm > m + kRescaleThresh) || stop);
        const float tmax = fmaxf(tm, pmax_s[(j & 1) * 128 + (1 - g) * 64 + h]);
        if (any && bar_softmax_or(flags[F_ABORT] != 0)) {
          ok = false;
          break;
        }
        if (ps) {
          m = tmax;
        } else if (any) {
          // bring O^T (all earlier PVs done: one thread issues them) to the new maxima
          float alpha = 1.f;
          if (tmax > m + kRescaleThresh) {
            alpha = m == -INFINITY ? 0.f : fast_exp2(m - tmax);
            m = tmax;
            lpart *= alpha;
          }
          if (g == 0 && lane < 16) alpha_s[h] = alpha;
          const bool got = tc::mbar_wait(bar(BAR_PV_DONE + (j - 1) % kSlots), ((j - 1) / kSlots) & 1, kWaitNs);
          if (bar_softmax_or(!got)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
#pragma unroll 1
          for (int blk = 0; blk < 4; ++blk) {
            uint32_t rr[32];
            const uint32_t ta = tmem + lane_base + kOCol + 64 * blk + 32 * g;
            tc::tmem_ld32(ta, rr);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha_s[32 * g + i]);
            tc::tmem_st32(ta, rr);
          }
          tc::tmem_wait_st();
        }
        // ---- P, this thread's 16 tokens of row h of P^T, into the page's rotary chunk ----
        {
          const float mu = m == -INFINITY ? 0.f : m;
          uint32_t w[8];
          float rs = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 a = add2(make_float2(s[2 * i], s[2 * i + 1]), make_float2(-mu, -mu));
            const float p0 = fast_exp2(a.x), p1 = fast_exp2(a.y);
            w[i] = bf16x2_of(p0, p1);
            rs += p0 + p1;  // the exact P: lse does not carry the operand rounding
          }
          lpart += rs;
          const uint32_t prow = page_base + (kChunks - 1) * kChunkBytes + h * 128;
          const int sw = h & 7;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(prow + (((2 * c16) ^ sw) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]));
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(prow + (((2 * c16 + 1) ^ sw) << 4)),
                       "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]));
        }
        if (nvis < kPageSize) {
          // value rows past the page's last token (all rows of a bad page id) become zeros
          // before PV reads them: their weights are 0, and 0 times a stale NaN would poison O
          for (int i = tid; i < (kPageSize - nvis) * 64; i += kSmThreads) {
            const int rrow = nvis + (i >> 6), u = i & 63;
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(
                             page_base + (u >> 3) * kChunkBytes + rrow * 128 + (u & 7) * 16),
                         "r"(0u));
          }
        }
        if (has_nodes) {
          // A NaN or an infinity in a node's entry is the scores' of the rows that see it; for
          // the others it would be 0 * NaN in PV, so 16-byte pieces with one become zeros.
          const int first = max((int)d.context, 0);
          for (int i = tid; i < (nvis - first) * 64; i += kSmThreads) {
            const int rrow = first + (i >> 6), u = i & 63;
            const uint32_t a = page_base + (u >> 3) * kChunkBytes + rrow * 128 + (u & 7) * 16;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
            if (bf16x2_not_finite(w[0]) || bf16x2_not_finite(w[1]) || bf16x2_not_finite(w[2]) ||
                bf16x2_not_finite(w[3]))
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(a), "r"(0u));
          }
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(BAR_P_FULL + slot));
        if (pe) {
          // ---- epilogue: O^T / l -> this piece's partial slot ----
          {
            const bool got = tc::mbar_wait(bar(BAR_O_FULL), (uint32_t)piece & 1, kWaitNs);
            if (bar_softmax_or(!got)) {
              ok = false;
              break;
            }
          }
          ++piece;
          tc::fence_after_sync();
          const float lh = lpart + __shfl_xor_sync(0xffffffffu, lpart, 16);
          if (lane < 16) lsum_s[g * 64 + h] = lh;
          int bad = 0;
          if (tid == 0) {
            bad = flags[F_PIECE_BAD];
            flags[F_PIECE_BAD] = 0;
          }
          bar_softmax();
          if (g == 0 && lane < 16) {
            // (a row without a node has whatever its q gives: it counts as empty)
            const float l = row_live ? lsum_s[h] + lsum_s[64 + h] : 0.f;
            linv_s[h] = l > 0.f ? p.kv_scale / l : 0.f;
            if (h < H)
              // (a NaN among the scores: lse = +inf, with which the merge makes the row NaN)
              p.ws.part_lse[(int64_t)d.slot * H + h] = l > 0.f    ? (m + log2f(l)) * kLn2
                                                       : l == 0.f ? -INFINITY
                                                                  : INFINITY;
          }
          if (tid == 0) p.ws.piece_err[d.slot] = bad;
          bar_softmax();
          // O^T lane = dim 128*blk + 32*(w%4) + lane; this warp writes rows 32g .. 32g+31
          if (32 * g < H) {
            float* out = p.ws.part_out + (int64_t)d.slot * H * kDLatent + 32 * q4 + lane;
#pragma unroll 1
            for (int blk = 0; blk < 4; ++blk) {
              uint32_t rr[32];
              tc::tmem_ld32(tmem + lane_base + kOCol + 64 * blk + 32 * g, rr);
              tc::tmem_wait_ld();
              float* o = out + (int64_t)(32 * g) * kDLatent + 128 * blk;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * g + i < H) o[(int64_t)i * kDLatent] = __uint_as_float(rr[i]) * linv_s[32 * g + i];
            }
          }
          if (j + 1 < pages) zero_o();
        }
      }
      if (!ok && tid == 0) abort_cta();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kQkWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

cudaError_t launch_kernel(const Bf16TreeParams& p, const CUtensorMap& kv_map, const CUtensorMap& q_map,
                          cudaStream_t stream) {
  static std::atomic<int> configured[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev].load()) {
    const cudaError_t e = cudaFuncSetAttribute(decode_bf16_tree_kernel,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(1);
  }
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.G);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_bf16_tree_kernel, p, kv_map, q_map);
}

}  // namespace

cudaError_t launch_decode_bf16_tree(const DecodeLaunch& d, cudaStream_t stream) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (encode == nullptr) {
    cudaDriverEntryPointQueryResult qr;
    void* fn = nullptr;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                     cudaEnableDefault, &qr);
    if (e != cudaSuccess || qr != cudaDriverEntryPointSuccess || fn == nullptr)
      return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  // pages as rows of 576 dims, and the query rows: boxes of 64 dims, a page or a tile high
  CUtensorMap kv_map, q_map;
  const cuuint64_t strides[1] = {(cuuint64_t)kDEntry * 2};
  const cuuint32_t estr[2] = {1, 1};
  auto map = [&](CUtensorMap* m, const void* base, int64_t rows, int high) {
    const cuuint64_t dims[2] = {(cuuint64_t)kDEntry, (cuuint64_t)rows};
    const cuuint32_t box[2] = {64, (cuuint32_t)high};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&kv_map, d.kv, (d.num_pages > 0 ? d.num_pages : 1) * kPageSize, kPageSize) ||
      !map(&q_map, d.q, (int64_t)d.batch * d.query_rows(), d.heads))
    return cudaErrorInvalidValue;
  Bf16TreeParams p;
  p.kv = d.kv;
  p.num_pages = d.num_pages;
  p.block_table = d.block_table;
  p.max_pages = d.max_pages;
  p.seq_lens = d.seq_lens;
  p.batch = d.batch;
  p.tiles = d.nq;
  p.tile_rows = d.heads;
  p.score_mul = d.score_mul;
  p.kv_scale = d.kv_scale;
  p.G = d.G;
  p.ws = d.ws;
  p.tree_mask = d.tree_mask;
  p.num_nodes = d.num_nodes;
  p.max_nodes = d.max_nodes;
  p.node_heads = d.node_heads;
  p.query_rows = d.query_rows();
  return launch_kernel(p, kv_map, q_map, stream);
}

}  // namespace mla
