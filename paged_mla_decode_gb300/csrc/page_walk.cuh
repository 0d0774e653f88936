// page_walk.cuh -- a decode CTA's walk over its pages: what its roles need to know of each
// page, and the cursor that finds it out (decode_fp8.cu, decode_bf16_tree.cu).
#pragma once

#include "mla_common.cuh"

namespace mla {
namespace {

// What every role needs to know about the CTA's j-th page, written by the TMA
// warp (the only planner walker) before it signals the page, read by the MMA and
// softmax warps after they have waited for it.
struct PageDesc {
  int32_t page;    // block-table entry
  int8_t valid;    // tokens of the row in this page (1..64)
  int8_t context;  // tree decode: how many of them come before the nodes (below 0: the
                   // page starts at node -context); 64 where all do
  int16_t flags;   // kDescPieceStart | kDescPieceEnd | kDescPageOk
  int32_t row;     // request row r = b * Q + j
  int32_t slot;    // partial slot of this piece
};
constexpr int16_t kDescPieceStart = 1, kDescPieceEnd = 2, kDescPageOk = 4;
constexpr int16_t kDescShared = 8;  // grouped decode: a shared-prefix page (informational)

// Cursor over a CTA's pages (one page per step). The row's partial slot and
// block-table offset are computed once per row: a step costs no division.
// `cta` is the worker index in the plan; for the grouped decode's plans the
// slot comes from the row table and `fork` picks the query row.
template <class P>
struct PageWalker {
  P plan;
  RowCursor cur;
  int64_t x, x_end, x_begin;
  int cta;         // this CTA's worker index in the plan
  int fork;        // grouped decode: the fork this CTA works for
  int slot;        // partial slot of the current row's piece in this CTA
  int qrow;        // query / output row of the current row
  int64_t bt_row;  // block-table offset of the current row's first page
  const int32_t* row_base;  // grouped decode: the row table
  const int32_t* row_np1;

  __device__ void init(const P& p, const RowCursor& c, int cta_index, int64_t xb, int64_t xe,
                       int fork_index = 0, const int32_t* rb = nullptr,
                       const int32_t* np1 = nullptr) {
    plan = p; cur = c; cta = cta_index; x = xb; x_begin = xb; x_end = xe;
    fork = fork_index; row_base = rb; row_np1 = np1;
    row_changed();
    settle();
  }
  __device__ void row_changed() {
    if constexpr (P::kGrouped) {
      qrow = plan.q_row(cur.r, fork);
      slot = __ldcg(row_base + qrow) + (plan.kind == 2 ? __ldcg(row_np1 + qrow) : 0) +
             (cta - plan.cta_of(cur.rt));
    } else {
      qrow = cur.r;
      slot = cur.base + (cta - plan.cta_of(cur.rt));
    }
    bt_row = plan.bt_base(cur.r);
  }
  __device__ void settle() {
    if (x < x_end && x == cur.rt + cur.t) {
      cursor_next_row(plan, cur);
      row_changed();
    }
  }
  __device__ int page_in_row() const { return (int)(x - cur.rt); }
  __device__ bool piece_start() const { return x == x_begin || x == cur.rt; }
  __device__ bool piece_end() const { return x + 1 == x_end || x + 1 == cur.rt + cur.t; }
  __device__ int valid_tokens() const { return min(kPageSize, cur.n - page_in_row() * kPageSize); }
  __device__ void next() { ++x; settle(); }
  // From a piece's first page: how many it has, and on to its last.
  __device__ int piece_pages() const {
    const int64_t row_end = cur.rt + cur.t;
    return (int)((x_end < row_end ? x_end : row_end) - x);
  }
  __device__ void to_piece_end(int pages) { x += pages - 1; }
  __device__ bool shared() const { return false; }
};

// Bit i: token i of the 16 from token `first` of a page on is one that a query row with
// node mask m sees, where the page's first `context` tokens come before the nodes.
__device__ __forceinline__ uint32_t tree_visible(uint64_t m, int context, int first) {
  const int s = context - first;  // of the 16, before the nodes
  if (s >= 16) return 0xffffu;
  if (s <= -64) return 0u;  // (behind the last possible node)
  const uint64_t nodes = s >= 0 ? m << s : m >> -s;
  return ((uint32_t)nodes | (s > 0 ? (1u << s) - 1u : 0u)) & 0xffffu;
}

}  // namespace
}  // namespace mla
