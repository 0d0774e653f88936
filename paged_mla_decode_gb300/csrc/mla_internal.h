// mla_internal.h -- host-side declarations shared by the library's .cu files.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "../../include/mla.h"

namespace mla {

// Typed views of a decode workspace (see WorkspaceLayout in mla_common.cuh).
struct DecodeWorkspace {
  unsigned* status;
  int32_t* row_base;
  int32_t* row_np;
  int32_t* row_np1;   // grouped decode: slots of each row's shared-prefix pieces
  int32_t* piece_err;
  float* part_lse;
  float* part_out;
  uint8_t* q_op;    // FP8 decode only: the split query operand of each row
  float* q_mul;     // FP8 decode only: score multiplier of each (row, head)
};

// Everything a decode kernel launch needs (validated by the caller).
struct DecodeLaunch {
  const __nv_bfloat16* q;
  const uint8_t* kv;
  int64_t num_pages;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seq_lens;
  int batch, nq, heads;
  bool bf16;         // cache holds bf16 (else e4m3 codes, or e2m1 pages)
  bool e2m1;         // cache holds e2m1 pages
  float score_mul;   // sm_scale * log2(e) * kv_scale
  float kv_scale;
  int G;             // CTAs launched
  DecodeWorkspace ws;
  // FP8 grouped decode only (else prefix_pages == nullptr): requests
  // [g * forks, (g + 1) * forks) share their first prefix_pages[g] pages
  int forks = 1;
  const int32_t* prefix_pages = nullptr;
  // tree decode only (else tree_mask == nullptr): nq is the tiles of a request, heads the
  // rows of a tile (see TreePlan), of which a request has max_nodes * node_heads in all
  const uint64_t* tree_mask = nullptr;
  const int32_t* num_nodes = nullptr;  // may be null
  int max_nodes = 0, node_heads = 0;
  int query_rows() const { return tree_mask ? max_nodes * node_heads : nq * heads; }  // of a request
};

// Split-KV decode on the tcgen05 tensor cores (decode_tc.cu); heads <= 64.
cudaError_t launch_decode_tensor_core(const DecodeLaunch& d, cudaStream_t stream);

// Split-KV decode with the e4m3 cache bytes as tensor-core operands
// (decode_fp8.cu); e4m3 and e2m1 caches, heads <= 64, num_pages * 64 < 2^31.
// Launches the query split (one pass per row into ws.q_op / ws.q_mul), then the
// decode kernel, which reads it.
cudaError_t launch_decode_fp8(const DecodeLaunch& d, cudaStream_t stream);

// Split-KV tree decode over a bf16 cache (decode_bf16_tree.cu); num_pages * 64 < 2^31.
cudaError_t launch_decode_bf16_tree(const DecodeLaunch& d, cudaStream_t stream);

// Merge the pieces written by a decode kernel into out (bf16) and lse (fp32);
// max_pieces_per_row is the number of decode CTAs (it sizes the staging), passes
// the number of plans that cut the rows (2 for the grouped decode). Row r, head h goes to
// output row r * heads + h; where `tiles` rows make a request of query_rows < tiles * heads
// output rows, to row (r / tiles) * query_rows + (r % tiles) * heads + h if there is one.
cudaError_t launch_combine_pieces(const DecodeWorkspace& ws, int rows, int heads, int passes,
                                  int max_pieces_per_row, __nv_bfloat16* out, float* lse,
                                  cudaStream_t stream, int tiles = 1, int query_rows = 0);

// Launch attribute that lets a kernel start while the previous kernel in the
// stream is finishing (programmatic dependent launch); kernels launched with it
// call griddep_wait() before their first global memory access.
inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// Number of SMs of the current device (cached per device).
int device_sm_count();

}  // namespace mla
