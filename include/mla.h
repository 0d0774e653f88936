/*
 * mla.h -- C ABI of the paged FP8 MLA decode library (libmla.so).
 *
 * Decode attention for multi-head latent attention (MLA) over a paged,
 * prefix-shareable latent KV cache, for one GPU (sm_103a).
 *
 * What the operations compute is described on these pages:
 *  - "How to serve trillions of tokens for trillion-parameter coding agents"
 *    (Modal), section "Tensor parallel was the best parallelism strategy for
 *    maximum interactivity": one cache entry per token and layer holds 576
 *    elements; section "First, understand the workload": the model keeps no
 *    distinct keys and values; section "Use custom speculative decoding ...":
 *    drafted tokens are verified in parallel without changing the target
 *    model's distribution.
 *  - "Smaller, faster, safer: running Kimi and GLM at scale" (Cloudflare),
 *    section "Quantizing the KV cache": the cache is FP8 e4m3 and the attention
 *    kernel converts values as it reads them; section "Protecting a shared KV
 *    cache": many requests read pages of one physical paged cache.
 *  - "vLLM x AgentX: Optimizing for Real-World Agentic Serving", section
 *    "Kimi K3": MLA has a single latent head shared by all query heads; partial
 *    attention outputs and their log-sum-exp statistics are merged with online
 *    softmax.
 *
 * Conventions shared by every entry point
 *  - Entry layout: 576 elements per token = 512 latent elements (the value,
 *    and the first 512 key elements) followed by 64 rotary key elements.
 *  - Cache layout: kv_pages[num_pages][page_size][576], row-major; one byte per
 *    element for MLA_KV_E4M3 (OCP E4M3: bias 7, max 448, no infinity), two
 *    (bfloat16) for MLA_KV_BF16. A token's slot is page_id * page_size + offset.
 *    page_size must be 64.
 *  - MLA_KV_E2M1 pages are MLA_E2M1_PAGE_BYTES contiguous bytes each:
 *      codes[18][64][16]  block b of token t (elements 32b .. 32b + 31), two e2m1
 *                         codes per byte, the even element in the low nibble;
 *      exps[9][64]        byte i of token t: the exponent nibbles of blocks 2i
 *                         (low) and 2i + 1 (high).
 *    An element's value is e2m1(code) * 2^(n - 8) * kv_scale, with e2m1 the
 *    values 0, 0.5, 1, 1.5, 2, 3, 4, 6 (code bit 3: sign) and n = 0..14 the
 *    block's nibble; n = 15 makes every element of the block NaN. Every such
 *    value is kv_scale times an e4m3 number, so the scale that suits an e4m3
 *    cache suits this one, and its kv_scale must lie in [2^-100, 2^100].
 *  - Pointers named "device" must point to device memory of the current CUDA
 *    device; all must be 16-byte aligned. The caller owns every buffer.
 *    The library allocates nothing and never synchronises the host: all work
 *    is enqueued on `stream` (NULL = the legacy default stream).
 *  - Arguments are checked on the host before anything is enqueued; a failed
 *    check returns MLA_ERR_INVALID_ARG or MLA_ERR_UNSUPPORTED and enqueues
 *    nothing. A failed launch returns MLA_ERR_CUDA.
 *  - Device-side problems (a block-table entry outside [0, num_pages), a
 *    sequence length outside [num_queries, max_pages * page_size]) never trap:
 *    the affected (request, draft) rows get out = 0 and lse = -inf, and a
 *    sticky bit is set in the status word at the start of the workspace
 *    (MLA_DEVICE_ERR_*), which the caller may read back at any time.
 *  - Entry points are re-entrant and keep no global state, with one
 *    exception: mla_decode_static_scratch keeps its scratch in one array per
 *    device, shared by all of its calls (see its declaration).
 *  - Stream order is kept: mla_decode's kernels are launched with programmatic
 *    dependent launch (they may become resident while the previous kernel in
 *    the stream finishes) but each waits for all earlier work in the stream to
 *    complete before its first memory access.
 */
#ifndef PAGED_MLA_DECODE_MLA_H_
#define PAGED_MLA_DECODE_MLA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MLA_API __attribute__((visibility("default")))
#else
#define MLA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st* mla_stream_t;

typedef enum mla_status {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1, /* a null pointer, a bad size, a misaligned buffer */
  MLA_ERR_UNSUPPORTED = 2, /* a shape the library has no kernel for */
  MLA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required */
  MLA_ERR_CUDA = 4         /* a CUDA runtime call or a launch failed */
} mla_status;

typedef enum mla_kv_dtype {
  MLA_KV_E4M3 = 0, /* FP8 e4m3 codes, one byte per element */
  MLA_KV_BF16 = 1, /* bfloat16, two bytes per element */
  MLA_KV_E2M1 = 2  /* FP4 e2m1 codes, 32 elements sharing a power of two (4.125 bits) */
} mla_kv_dtype;

#define MLA_D_LATENT 512
#define MLA_D_ROPE 64
#define MLA_D_ENTRY 576
#define MLA_PAGE_SIZE 64
#define MLA_MAX_QUERIES 4
#define MLA_E2M1_BLOCK 32         /* elements that share an exponent in an MLA_KV_E2M1 cache */
#define MLA_E2M1_PAGE_BYTES 19008 /* bytes of an MLA_KV_E2M1 page of 64 tokens */

/* Bits of the device status word (first 4 bytes of the decode workspace). */
#define MLA_DEVICE_ERR_BAD_PAGE 0x1u   /* a block-table entry outside the cache */
#define MLA_DEVICE_ERR_BAD_LENGTH 0x2u /* seq_len < num_queries or > max_pages*page_size */
#define MLA_DEVICE_ERR_TIMEOUT 0x4u    /* an internal pipeline wait ran out (2 s); results invalid */

/* Version of this ABI (increments on any incompatible change). */
MLA_API int mla_abi_version(void);

/* Static, human-readable name of a status code; never NULL. */
MLA_API const char* mla_status_string(int status);

/*
 * mla_kv_append -- write new tokens' latent entries into their cache slots.
 *
 * The cache-write side of "Quantizing the KV cache" (Cloudflare page above):
 * for each token t < num_tokens with slot_mapping[t] >= 0,
 *   MLA_KV_E4M3: kv_pages[slot][d] = e4m3( x[t][d] / kv_scale ), rounded to
 *                nearest with ties to even, of the exact quotient, and
 *                saturated to +-448 (NaN stays NaN), where x[t][0:512] =
 *                latent[t], x[t][512:576] = rope[t];
 *   MLA_KV_BF16: kv_pages[slot][d] = x[t][d] (a copy; kv_scale must be 1);
 *   MLA_KV_E2M1: per block of 32 elements with a = max |x|: n - 8 is the smallest
 *                power in -8 .. 6 with a <= 7 * 2^(n - 8) * kv_scale (6 if there
 *                is none), and each code is the exact quotient
 *                x / (2^(n - 8) * kv_scale) rounded to the nearest e2m1 value,
 *                ties to the even code, saturated at +-6 (between 6 and 7 the
 *                error is at most the half step of 4 .. 6, which a larger power
 *                would double). Infinities saturate; a block that holds a NaN
 *                gets n = 15 and zero codes.
 * Slots with slot_mapping[t] < 0 are skipped (padding tokens).
 *
 * latent       device, bf16 [num_tokens][512], row-major
 * rope         device, bf16 [num_tokens][64], row-major
 * slot_mapping device, int32 [num_tokens]; each must be -1 or lie in
 *              [0, num_pages * page_size) (entries beyond it are skipped and
 *              nothing else is reported; validate on the host if needed)
 * kv_pages     device, the cache (see layout above); written in place
 * kv_scale     per-tensor scale, finite and > 0
 * Two tokens naming the same slot race; writing into a page that other
 * requests share is the caller's error.
 */
MLA_API mla_status mla_kv_append(const void* latent, const void* rope, const int32_t* slot_mapping,
                         int64_t num_tokens, void* kv_pages, int64_t num_pages, int page_size,
                         int kv_dtype, float kv_scale, mla_stream_t stream);

/*
 * mla_decode_workspace_size -- bytes of workspace mla_decode needs.
 *
 * num_ctas is the number of worker CTAs the caller will pass to mla_decode
 * (0 = the default, one per SM of the current device). Returns 0 for an
 * invalid shape.
 */
MLA_API size_t mla_decode_workspace_size(int batch, int num_queries, int num_heads, int num_ctas);

/*
 * mla_decode -- attention of the new query tokens over each request's pages.
 *
 * For request b < batch, draft j < num_queries and head h < num_heads, with
 * L = seq_lens[b] counting the cached tokens including the num_queries drafts
 * just appended, draft j sees positions t < n_j = L - num_queries + j + 1:
 *   K[t]  = value(kv_pages[block_table[b][t / page_size]][t % page_size]) * kv_scale
 *   s_t   = sm_scale * sum_{d<576} q[b][j][h][d] * K[t][d]
 *   lse   = ln sum_t exp(s_t)
 *   out   = sum_t exp(s_t - lse) * K[t][0:512]
 * (natural logarithm; s includes sm_scale). The work is split into pieces of
 * equal token count over num_ctas CTAs (split-KV); each piece yields a partial
 * (out, lse) that a second kernel merges by log-sum-exp ("vLLM x AgentX",
 * section "Kimi K3"), so one call fills all SMs even at batch 1.
 *
 * Arithmetic: for an e4m3 cache the cache bytes themselves are the tensor-core
 * operands (tcgen05 kind::f8f6f4); q is scaled per head by a power of two and
 * split into two e4m3 terms (exact for bf16 q down to 2^-10 of the head's
 * largest element); accumulation is fp32. The softmax weights P = 2^(s - m + 6)
 * (s in log2 units, m a running maximum) are split into an e4m3 and an e5m2
 * term: relative error at most 2^-7 for P >= 2^-6, coarser below, and P below
 * about 2^-17 drops out of `out` (the normaliser sums the exact P). m follows
 * each 64-token page's maximum within [-6, +2.8] (a page further below lowers
 * m, unless the weight accumulated so far exceeds 2^28 times the page's
 * largest), so every page's largest P lies in [1, 448]; what a page loses is
 * confined to its tokens below 2^-6 of its largest weight. Each piece of the
 * split (one per CTA) has its own maximum; pieces merge in fp32. An e2m1 cache
 * is expanded to e4m3 codes in shared memory as its pages arrive, which is
 * exact, and then takes the same arithmetic. For a bf16 cache both contractions
 * use bf16 operands (kind::f16). With every cache a NaN among a head's visible
 * scores (from a cached NaN, or from a NaN or an infinity in its query) makes
 * that row NaN, out and lse.
 *
 * q           device, bf16 [batch][num_queries][num_heads][576]
 * kv_pages    device, the cache; num_pages pages of page_size (= 64) tokens
 * block_table device, int32 [batch][max_pages]; entries past a request's last
 *             page are never read
 * seq_lens    device, int32 [batch]
 * num_heads   16, 32 or 64 (UNSUPPORTED otherwise)
 * num_queries 1..4
 * sm_scale, kv_scale  finite; kv_scale > 0 (use 1 for MLA_KV_BF16 caches)
 * num_ctas    worker CTAs (0 = one per SM); must match the value the
 *             workspace was sized for
 * workspace   device, at least mla_decode_workspace_size(batch, num_queries,
 *             num_heads, num_ctas) bytes, zero-filled before its first use;
 *             every call leaves it ready for the next (status word aside).
 *             Calls that share a workspace must be stream-ordered.
 * out         device, bf16 [batch][num_queries][num_heads][512]
 * lse         device, fp32 [batch][num_queries][num_heads]
 */
MLA_API mla_status mla_decode(const void* q, const void* kv_pages, int64_t num_pages, int page_size,
                      int kv_dtype, const int32_t* block_table, int max_pages,
                      const int32_t* seq_lens, int batch, int num_queries, int num_heads,
                      float sm_scale, float kv_scale, int num_ctas, void* workspace,
                      size_t workspace_bytes, void* out, float* lse, mla_stream_t stream);

/*
 * mla_decode_grouped -- mla_decode for groups of requests that share a prefix.
 *
 * Subagent sessions fork from a parent context ("vLLM x AgentX: Optimizing for
 * Real-World Agentic Serving", section "Characterizing agentic workloads: a
 * second look") and then read the pages of one physical paged cache ("Smaller,
 * faster, safer: running Kimi and GLM at scale", section "Protecting a shared KV
 * cache"). Requests [g * forks, (g + 1) * forks) form group g, and their first
 * prefix_pages[g] logical pages are the same physical pages; the kernel reads
 * those page ids from the group's first request. The results are mla_decode's
 * on the same arguments (same arithmetic and tolerance); what changes is how
 * the work is cut: each shared page is worked by `forks` CTAs at once, one per
 * fork, so the group reads it from HBM once (the other forks' reads hit L2),
 * while the tokens after the prefix are split as in mla_decode.
 *
 * forks         requests per group; 1 <= forks <= CTAs and batch % forks == 0
 * prefix_pages  device, int32 [batch / forks]. A request whose group prefix is
 *               outside [0, max_pages] pages or longer than L - num_queries + 1
 *               tokens (draft 0 must see the whole prefix) is treated like a
 *               bad length: out = 0, lse = -inf, MLA_DEVICE_ERR_BAD_LENGTH.
 * workspace     at least mla_decode_grouped_workspace_size(batch, num_queries,
 *               num_heads, num_ctas) bytes, zero-filled before its first use.
 * kv_dtype      MLA_KV_E4M3 or MLA_KV_E2M1 (MLA_ERR_UNSUPPORTED otherwise).
 * Other arguments as mla_decode.
 */
MLA_API size_t mla_decode_grouped_workspace_size(int batch, int num_queries, int num_heads,
                                                 int num_ctas);
MLA_API mla_status mla_decode_grouped(const void* q, const void* kv_pages, int64_t num_pages,
                                      int page_size, int kv_dtype, const int32_t* block_table,
                                      int max_pages, const int32_t* seq_lens, int batch,
                                      int num_queries, int num_heads, int forks,
                                      const int32_t* prefix_pages, float sm_scale,
                                      float kv_scale, int num_ctas, void* workspace,
                                      size_t workspace_bytes, void* out, float* lse,
                                      mla_stream_t stream);

/*
 * mla_decode_tree -- attention of a tree of drafted tokens.
 *
 * A drafter may propose several continuations of a request: a tree whose nodes are
 * verified in parallel without changing the target model's distribution ("How to
 * serve trillions of tokens for trillion-parameter coding agents", section "Use
 * custom speculative decoding ..."). The n = num_nodes[b] nodes of request b are its
 * last n cached tokens, in node order (node 0 the last sampled token, the others
 * drafts behind it); L = seq_lens[b] counts them. Node j sees the L - n tokens of the
 * context and each node i < n whose bit i is set in tree_mask[b][j], for a tree its
 * ancestors and itself; any other set is as good, and a row that sees no token gets
 * out = 0, lse = -inf. K, s, out and lse as in mla_decode, over the tokens that the
 * node sees. A chain of drafts is the mask 2^(j + 1) - 1.
 *
 * The max_nodes * num_heads query rows of a request are cut into tiles of 64, whatever
 * nodes they belong to; a tile's rows share each page that is read. Arithmetic as
 * mla_decode's; so a NaN in an entry makes the rows that see it NaN, and no others. A
 * cached bf16 infinity does so too, except in rows whose score of it is -inf: there the
 * entry has no weight in out or lse, but the latent dims of out at which a context token
 * (not a node) holds the infinity may be NaN, as 0 times it.
 *
 * tree_mask   device, uint64 [batch][max_nodes]
 * num_nodes   device, int32 [batch]; NULL: max_nodes each. Rows j >= num_nodes[b] get
 *             out = 0, lse = -inf. A request with num_nodes[b] outside
 *             [0, max_nodes] or a length outside [num_nodes[b], max_pages * 64] is
 *             a bad length (MLA_DEVICE_ERR_BAD_LENGTH, out = 0, lse = -inf).
 * max_nodes   1 .. MLA_MAX_TREE_NODES
 * q           device, bf16 [batch][max_nodes][num_heads][576]
 * out         device, bf16 [batch][max_nodes][num_heads][512]
 * lse         device, fp32 [batch][max_nodes][num_heads]
 * workspace   at least mla_decode_tree_workspace_size(batch, max_nodes, num_heads,
 *             num_ctas) bytes, zero-filled before its first use.
 * Other arguments as mla_decode, num_heads and the cache types too.
 */
#define MLA_MAX_TREE_NODES 64
MLA_API size_t mla_decode_tree_workspace_size(int batch, int max_nodes, int num_heads,
                                              int num_ctas);
MLA_API mla_status mla_decode_tree(const void* q, const void* kv_pages, int64_t num_pages,
                                   int page_size, int kv_dtype, const int32_t* block_table,
                                   int max_pages, const int32_t* seq_lens,
                                   const uint64_t* tree_mask, const int32_t* num_nodes,
                                   int batch, int max_nodes, int num_heads, float sm_scale,
                                   float kv_scale, int num_ctas, void* workspace,
                                   size_t workspace_bytes, void* out, float* lse,
                                   mla_stream_t stream);

/*
 * mla_decode_f16_operands -- mla_decode with 16-bit tensor-core operands.
 *
 * Same arguments, contract and results (within the same tolerance) as
 * mla_decode. For an e4m3 cache the pages are widened to f16 in shared memory
 * as they are read (the FP8 cache of "Smaller, faster, safer: running Kimi and
 * GLM at scale", section "Quantizing the KV cache", converted on load) and both
 * contractions use kind::f16 with q and the softmax weights in f16; for a bf16
 * cache it is mla_decode; MLA_KV_E2M1 is refused (MLA_ERR_UNSUPPORTED). It
 * exists to measure what reading the FP8 bytes as operands saves; it has no
 * counterpart on the pages.
 */
MLA_API mla_status mla_decode_f16_operands(const void* q, const void* kv_pages, int64_t num_pages,
                                   int page_size, int kv_dtype, const int32_t* block_table,
                                   int max_pages, const int32_t* seq_lens, int batch,
                                   int num_queries, int num_heads, float sm_scale,
                                   float kv_scale, int num_ctas, void* workspace,
                                   size_t workspace_bytes, void* out, float* lse,
                                   mla_stream_t stream);

/*
 * mla_decode_combine -- merge partial attention results by log-sum-exp.
 *
 * The merge of "vLLM x AgentX", section "Kimi K3" (partial outputs and LSE
 * statistics combined with online softmax), for partials produced elsewhere
 * (for example one per sequence shard). For each row r < num_rows:
 *   lse[r] = ln sum_s exp(part_lse[s][r])
 *   out[r] = sum_s exp(part_lse[s][r] - lse[r]) * part_out[s][r][0:512]
 * A part with part_lse = -inf contributes nothing; if all are -inf the row
 * gets out = 0 and lse = -inf.
 * A part with part_lse = NaN (a NaN row of mla_decode) makes the row NaN.
 *
 * part_out  device, fp32 [num_parts][num_rows][512] (normalised partials)
 * part_lse  device, fp32 [num_parts][num_rows]
 * out       device, bf16 [num_rows][512]
 * lse       device, fp32 [num_rows]
 */
MLA_API mla_status mla_decode_combine(const float* part_out, const float* part_lse, int num_parts,
                              int64_t num_rows, void* out, float* lse, mla_stream_t stream);

/*
 * mla_kv_gather -- read cached entries back as bfloat16 rows.
 *
 * The read side of mla_kv_append ("Smaller, faster, safer: running Kimi and GLM
 * at scale", section "Quantizing the KV cache": values are converted back as
 * they are read), for callers that need the entries themselves, such as a
 * prefill chunk over a cached context. Row r with cu_tokens[b] <= r <
 * cu_tokens[b + 1] receives token starts[b] + r - cu_tokens[b] of request b:
 *   latent[r][0:512], rope[r][0:64] = bf16( value(code) * kv_scale )
 * the product in fp32, rounded to bf16 (a bf16 cache is copied). A token beyond
 * its block-table row or in a page outside the cache gives a row of zeros. Rows
 * from cu_tokens[batch] on are left as they were.
 *
 * kv_pages, num_pages, page_size, kv_dtype, kv_scale  as for mla_kv_append
 * block_table device, int32 [batch][max_pages]
 * starts      device, int32 [batch]; NULL: every range starts at token 0
 * cu_tokens   device, int32 [batch + 1], ascending
 * num_tokens  rows of latent and rope; ranges beyond it are cut
 * latent      device, bf16 [num_tokens][512] (written)
 * rope        device, bf16 [num_tokens][64] (written)
 */
MLA_API mla_status mla_kv_gather(const void* kv_pages, int64_t num_pages, int page_size,
                                 int kv_dtype, float kv_scale, const int32_t* block_table,
                                 int max_pages, const int32_t* starts, const int32_t* cu_tokens,
                                 int batch, int64_t num_tokens, void* latent, void* rope,
                                 mla_stream_t stream);

/*
 * mla_kv_alloc -- extend requests by new tokens: pages, block tables, slots.
 *
 * The page allocator's side of a step, on the device, from the requests'
 * lengths (see mla_kv_check for the page tags). For request b = 0, 1, ... in
 * order, with L = seq_lens[b] cached tokens, n = new_tokens[b] and
 * h = pages_held[b] block-table entries in use (pages kept from rejected drafts
 * among them: h >= ceil(L / 64)):
 *   cu_tokens[b + 1] = cu_tokens[b] + max(n, 0), cu_tokens[0] = 0;
 *   it takes max(0, ceil((L + n) / 64) - h) pages off the end of the free list,
 *   the last one first, and appends them to its block-table row; with tags,
 *   page_tags[p] += 1 for each and expected_tags beside the entry = the new tag;
 *   slot_mapping[cu_tokens[b] + i] = slot of token L + i, for mla_kv_append;
 *   seq_lens_out[b] = L + n, pages_held_out[b] = h + pages taken.
 * A refused request takes no page; its slots are -1, seq_lens_out[b] = -1 and
 * request_status[b] says why:
 *   MLA_KV_ALLOC_BAD_LENGTH  L < 0 (as mla_kv_check marks a failed request),
 *                            n < 0, h outside [ceil(L / 64), max_pages];
 *   MLA_KV_ALLOC_TABLE_FULL  L + n tokens need more than max_pages pages;
 *   MLA_KV_ALLOC_SLOTS_FULL  its rows end beyond num_slots;
 *   MLA_KV_ALLOC_NO_PAGES    the pages asked for so far, its own included,
 *                            exceed the free list (so does every later request
 *                            that needs a page).
 * Slots from cu_tokens[batch] on are -1 (padding, which mla_kv_append skips). A
 * free-list entry outside [0, num_pages) reaches the block table as it is, where
 * mla_kv_check and mla_decode report it; its slots are -1.
 *
 * seq_lens, new_tokens, pages_held  device, int32 [batch]
 * free_pages      device, int32 [free_capacity]; the first *free_count are free
 * free_count      device, int32; taken as 0 below 0, free_capacity above it
 * block_table     device, int32 [batch][max_pages], updated in place
 * page_tags       device, uint32 [num_pages], updated in place; or NULL
 * expected_tags   device, uint32 [batch][max_pages], updated in place; NULL
 *                 exactly if page_tags is (without requests or pages either may be)
 * seq_lens_out, pages_held_out  device, int32 [batch]
 * free_count_out  device, int32
 *                 Each output of these three may be the same buffer as its
 *                 input, so that a captured step can be replayed. (The length of a
 *                 refused request is then gone: keep seq_lens apart, or a copy,
 *                 where refused requests are to be tried again.)
 * cu_tokens       device, int32 [batch + 1] (saturates at 2^31 - 1)
 * slot_mapping    device, int32 [num_slots]
 * request_status  device, uint32 [batch]
 * Pointers need 4-byte alignment here. A page named twice by the free list, or
 * free and held, is the caller's error. Pages come back to the list by the
 * caller's own writes: a finished request's block-table entries, behind the
 * first *free_count.
 */
#define MLA_KV_ALLOC_BAD_LENGTH 0x1u
#define MLA_KV_ALLOC_TABLE_FULL 0x2u
#define MLA_KV_ALLOC_SLOTS_FULL 0x4u
#define MLA_KV_ALLOC_NO_PAGES 0x8u
MLA_API mla_status mla_kv_alloc(const int32_t* seq_lens, const int32_t* new_tokens, int batch,
                                int page_size, const int32_t* pages_held,
                                const int32_t* free_pages, const int32_t* free_count,
                                int64_t free_capacity, int64_t num_pages, int32_t* block_table,
                                int max_pages, uint32_t* page_tags, uint32_t* expected_tags,
                                int32_t* seq_lens_out, int32_t* pages_held_out,
                                int32_t* free_count_out, int32_t* cu_tokens,
                                int32_t* slot_mapping, int64_t num_slots,
                                uint32_t* request_status, mla_stream_t stream);

/*
 * mla_verify_drafts -- accept or reject drafted tokens, sample the next one.
 *
 * The end of a speculative step ("How to serve trillions of tokens for
 * trillion-parameter coding agents", section "Use custom speculative decoding
 * ...": drafts are verified in parallel without changing the target model's
 * distribution). For request b with k = num_drafts[b] drafts x_0 .. x_{k-1},
 * p_j = target_probs[b][j], q_j = draft_probs[b][j] and u = uniforms[b]:
 *   draft j is kept while u_j * q_j(x_j) < p_j(x_j) (and every earlier one was);
 *   a = num_accepted[b] = the number kept;
 *   the next token is drawn from max(p_a - q_a, 0) if a < k (from p_a if that is
 *   zero everywhere), from p_k if a = k: the smallest i with
 *   w_0 + .. + w_i > uniforms[b][max_drafts] * (w_0 + .. + w_{vocab-1});
 *   out_tokens[b] = x_0 .. x_{a-1}, the next token, then -1;
 *   seq_lens_out[b] = seq_lens[b] - (k - a), the cached tokens that stay
 *   (seq_lens[b] counts the k + 1 queries of the step).
 * A call of mla_decode has max_drafts + 1 queries for every request, the last of
 * them the last cached token. So a request with k < max_drafts drafts is cached
 * and decoded with max_drafts + 1 new tokens, anything behind its drafts, which
 * gives row j of target_probs the output of query j; here it passes the length
 * without that padding, mla_decode's less max_drafts - k. The padding's slots
 * are the next step's.
 * With draft_probs NULL, q_j puts all its weight on x_j: u_j < p_j(x_j), and the
 * rest is p_a without x_a. A draft outside [0, vocab) is rejected. If all
 * weights are zero the next token is -1. A request with k outside
 * [0, max_drafts] or a negative length is left out: out_tokens[b] = -1
 * throughout, num_accepted[b] = -1, seq_lens_out[b] = seq_lens[b].
 *
 * Arithmetic: probabilities are taken within [0, 1] (NaN as 0), uniforms within
 * [0, 1 - 2^-24] (NaN as 0). The acceptance test is exact; weights are summed as
 * integers in units of 2^-60 (a probability below 2^-37 is rounded to them),
 * so the result does not depend on the order of the sum. A row's probabilities
 * must sum to less than 16 (beyond it the sums wrap: some token, or -1).
 *
 * target_probs  device, [batch][max_drafts + 1] rows of `vocab` probabilities,
 *               target_stride >= vocab elements apart
 * draft_probs   device, [batch][max_drafts] rows, draft_stride apart; or NULL
 * prob_dtype    MLA_PROB_F32 or MLA_PROB_BF16, of both
 * draft_tokens  device, int32 [batch][max_drafts] (may be NULL if max_drafts = 0)
 * uniforms      device, fp32 [batch][max_drafts + 1]
 * num_drafts    device, int32 [batch]; NULL: max_drafts each
 * seq_lens      device, int32 [batch]; may be NULL (then seq_lens_out is too)
 * max_drafts    0 .. MLA_MAX_DRAFTS
 * out_tokens    device, int32 [batch][max_drafts + 1]
 * num_accepted  device, int32 [batch]
 * seq_lens_out  device, int32 [batch]; may be seq_lens, or NULL
 * Pointers need the alignment of their elements here.
 */
#define MLA_MAX_DRAFTS 31
typedef enum mla_prob_dtype { MLA_PROB_F32 = 0, MLA_PROB_BF16 = 1 } mla_prob_dtype;
MLA_API mla_status mla_verify_drafts(const void* target_probs, int64_t target_stride,
                                     const void* draft_probs, int64_t draft_stride,
                                     int prob_dtype, const int32_t* draft_tokens,
                                     const float* uniforms, const int32_t* num_drafts,
                                     const int32_t* seq_lens, int batch, int max_drafts,
                                     int vocab, int32_t* out_tokens, int32_t* num_accepted,
                                     int32_t* seq_lens_out, mla_stream_t stream);

/*
 * mla_logits_to_probs -- logits to the probabilities that a request samples from.
 *
 * What stands between the target model's logits and the verification of drafts, which
 * must not change the model's distribution ("How to serve trillions of tokens for
 * trillion-parameter coding agents", section "Use custom speculative decoding ..."): each
 * request's own settings, for mla_verify_drafts (rows = drafts + 1) and mla_verify_tree
 * (rows = nodes), and for a drafter's logits alike. For row j of request b, token v, with
 * n(v) = max(token_counts[b][v], 0) + the number of drafts i >= 1 with bit i of
 * tree_mask[b][j] and node_tokens[b][i] = v (node 0's token is among the counted):
 *   if n(v) > 0 or v is in the prompt: x = x > 0 ? x / repetition : x * repetition;
 *   if n(v) > 0: x = x - frequency * n(v) - presence;
 *   x = x + biases[b][i] for every i with bias_tokens[b][i] = v;
 *   x = -inf where bit v of allowed[b][j] is 0, and where x is NaN;
 *   p(v) = exp((x(v) - max x) / temperature) / sum.
 * A temperature that is not above 0 puts all weight on the maximum, the lowest token of
 * equal ones; tokens at +inf share the weight; a row without a token above -inf is 0
 * throughout (the verifications then give the token -1). Arithmetic in fp32 (a logit that leaves
 * its range is an infinity), rounded once.
 *
 * logits        device, [batch][rows] rows of `vocab`, logit_stride >= vocab elements apart
 * probs         device, likewise, prob_stride apart; may be `logits` (same type and stride)
 * logit_dtype, prob_dtype  MLA_PROB_F32 or MLA_PROB_BF16
 * vocab         1 .. MLA_MAX_PROBS_VOCAB (UNSUPPORTED beyond: a byte a token is kept on chip)
 * temperature   device, fp32 [batch]; NULL: 1
 * num_rows      device, int32 [batch]; rows j >= num_rows[b] are left as they were; NULL: none
 * node_tokens   device, int32 [batch][rows]; NULL exactly if tree_mask is (then no drafts
 *               count). Tokens outside the vocabulary count for nothing.
 * tree_mask     device, uint64 [batch][rows], rows <= MLA_MAX_TREE_NODES; 8-byte aligned. A
 *               chain of drafts is 2^(j + 1) - 1.
 * token_counts  device, int32 [batch][vocab]; NULL: 0
 * prompt_mask   device, uint32 [batch][ceil(vocab / 32)], bit v % 32 of word v / 32; NULL: 0
 * repetition, frequency, presence  device, fp32 [batch]; NULL: 1, 0, 0
 * bias_tokens   device, int32 [batch][num_biases]; entries outside the vocabulary (-1:
 *               padding) are skipped; the same token may come twice
 * biases        device, fp32 [batch][num_biases]
 * num_biases    0 .. MLA_MAX_BIASES (UNSUPPORTED beyond)
 * allowed       device, uint32 [batch][rows][ceil(vocab / 32)]; NULL: everything
 * Other pointers need the alignment of their elements here.
 */
#define MLA_MAX_PROBS_VOCAB 393216
#define MLA_MAX_BIASES 1024
MLA_API mla_status mla_logits_to_probs(
    const void* logits, int64_t logit_stride, int logit_dtype, void* probs, int64_t prob_stride,
    int prob_dtype, int batch, int rows, int vocab, const float* temperature,
    const int32_t* num_rows, const int32_t* node_tokens, const uint64_t* tree_mask,
    const int32_t* token_counts, const uint32_t* prompt_mask, const float* repetition,
    const float* frequency, const float* presence, const int32_t* bias_tokens, const float* biases,
    int num_biases, const uint32_t* allowed, mla_stream_t stream);

/*
 * mla_verify_tree -- walk down a tree of drafts, sample the token behind it.
 *
 * mla_verify_drafts for a tree. The parent of node i > 0 is the last node before i that
 * bits of tree_mask[b][i] name (its last ancestor); a node without one is never reached.
 * With p_v = target_probs[b][v], q_v = draft_probs[b][v] (which v's children were drawn
 * from, independently of each other), x_i = node_tokens[b][i], u = uniforms[b], from node
 * v = 0 on, R = p_v and W = 1:
 *   the children i of v are tried in order: i is kept if u_i * q_v(x_i) * W < R(x_i);
 *   then v = i, R = p_i, W = 1. Else R = max(R - W * q_v, 0) and W = the sum of R.
 *   When no child is left: the next token is drawn from R (from p_v if R is 0 everywhere):
 *   the smallest token whose running sum exceeds u_0 times the sum.
 * With draft_probs NULL a child's token was certain: it is kept if u_i * W < R(x_i), else
 * W = max(W - R(x_i), 0) and R(x_i) = 0. A draft outside [0, vocab) is rejected. For a chain
 * this is mla_verify_drafts' rule.
 *   out_tokens[b] = the kept drafts' tokens, the next token (-1 if all weights are
 *   zero), then -1; path[b] = 0, the kept nodes, then -1;
 *   num_accepted[b] = a, the number of kept drafts;
 *   seq_lens_out[b] = seq_lens[b] - n + a + 1, the length after mla_kv_compact;
 *   token_counts[b][t] += 1 for every token t of out_tokens[b] that is not -1.
 * A request with n = num_nodes[b] outside [1, max_nodes] or seq_lens[b] < n is left out:
 * out_tokens[b] = path[b] = -1 throughout, num_accepted[b] = -1, seq_lens_out[b] =
 * seq_lens[b], token_counts[b] as it was.
 *
 * Arithmetic as in mla_verify_drafts: weights are summed as integers in units of 2^-60.
 * After a node's second rejection R = max(p_v - c * q_v, 0) for the sum c of its Ws, c
 * rounded to fp32 and R too. A row's probabilities must sum to less than 16 (beyond it the
 * sums wrap: some child or none is kept, some token or -1 follows).
 *
 * target_probs, draft_probs  device, [batch][max_nodes] rows of `vocab` probabilities,
 *               target_stride, draft_stride elements apart; rows >= num_nodes[b] and a
 *               leaf's row of draft_probs are never read
 * node_tokens   device, int32 [batch][max_nodes]; node 0's is not looked at
 * tree_mask     device, uint64 [batch][max_nodes], 8-byte aligned
 * uniforms      device, fp32 [batch][max_nodes]: u_0 for the sample, u_i for node i
 * num_nodes     device, int32 [batch]; NULL: max_nodes each
 * seq_lens      device, int32 [batch], lengths with all nodes; may be NULL (then
 *               seq_lens_out is too)
 * max_nodes     1 .. MLA_MAX_TREE_NODES
 * out_tokens, path  device, int32 [batch][max_nodes]
 * num_accepted  device, int32 [batch]
 * seq_lens_out  device, int32 [batch]; may be seq_lens, or NULL
 * token_counts  device, int32 [batch][vocab], as mla_logits_to_probs takes them; or NULL
 * Other pointers need the alignment of their elements here.
 */
MLA_API mla_status mla_verify_tree(const void* target_probs, int64_t target_stride,
                                   const void* draft_probs, int64_t draft_stride, int prob_dtype,
                                   const int32_t* node_tokens, const uint64_t* tree_mask,
                                   const float* uniforms, const int32_t* num_nodes,
                                   const int32_t* seq_lens, int batch, int max_nodes, int vocab,
                                   int32_t* out_tokens, int32_t* path, int32_t* num_accepted,
                                   int32_t* seq_lens_out, int32_t* token_counts,
                                   mla_stream_t stream);

/*
 * mla_kv_compact -- move the kept nodes' entries behind the context.
 *
 * After mla_verify_tree the kept nodes' entries stand among those of rejected ones
 * (drafts are verified in parallel: section "Use custom speculative decoding ..." of the
 * page above). For request b with a = num_accepted[b] >= 1, and
 * base = seq_lens[b] - a - 1 the tokens of its context:
 *   the entry of token base + path[b][i] goes to token base + i, i = 1 .. a,
 * in each of num_layers caches with the same block table, as stored (bit for bit). All
 * entries are read before one is written. A source outside [base, base + max_nodes) or
 * beyond the block-table row, or a source or destination in no page of the cache, is
 * skipped. Requests with a < 1, a >= max_nodes, or a length outside
 * [a + 1, max_pages * 64] are left as they are. The block table must still name the pages
 * of the rejected nodes.
 *
 * kv_pages      device, the first layer's pages (layout by kv_dtype); written in place
 * layer_stride  bytes from one layer's pages to the next's, a multiple of 16 and at least
 *               a layer's pages (not looked at with one layer)
 * num_layers    0 .. 65535
 * seq_lens      device, int32 [batch], lengths after verification (its seq_lens_out)
 * path          device, int32 [batch][max_nodes]
 * num_accepted  device, int32 [batch]
 * Other arguments as mla_decode_tree; index arrays need 4-byte alignment.
 */
MLA_API mla_status mla_kv_compact(void* kv_pages, int num_layers, int64_t layer_stride,
                                  int64_t num_pages, int page_size, int kv_dtype,
                                  const int32_t* block_table, int max_pages,
                                  const int32_t* seq_lens, const int32_t* path,
                                  const int32_t* num_accepted, int batch, int max_nodes,
                                  mla_stream_t stream);

/*
 * mla_kv_check -- integrity check of requests' page mappings before decode.
 *
 * The check of "Smaller, faster, safer: running Kimi and GLM at scale",
 * section "Protecting a shared KV cache": every physical page carries a tag
 * that the page allocator changes whenever it hands the page out again; each
 * request keeps, beside its block-table entries, the tags its pages had when it
 * was given them; before decode reads the cache the two are compared, and a
 * request with any mismatch is aborted instead of reading another request's
 * data. It is a separate batch pass, not part of the attention kernel.
 *
 * For request b < batch with L = seq_lens[b], over its used logical pages
 * j < ceil(L / page_size), with p = block_table[b][j]:
 *   MLA_KV_CHECK_PAGE_RANGE   if p < 0 or p >= num_pages;
 *   MLA_KV_CHECK_TAG_MISMATCH if page_tags[p] != expected_tags[b][j];
 *   MLA_KV_CHECK_BAD_LENGTH   (and no page looked at) if L < 0 or
 *                             L > max_pages * page_size.
 * request_status[b] = OR of the bits (0 = the request passed);
 * checked_seq_lens[b] = L if it passed, else -1. Passing checked_seq_lens to
 * mla_decode as seq_lens aborts the failed requests there: each of their rows
 * gets out = 0 and lse = -inf (and MLA_DEVICE_ERR_BAD_LENGTH in the workspace
 * status word) and none of their pages is read.
 *
 * page_tags        device, uint32 [num_pages] (may be NULL if num_pages == 0)
 * block_table      device, int32 [batch][max_pages]; entries past a request's
 *                  used pages are not read
 * expected_tags    device, uint32 [batch][max_pages], beside block_table
 * seq_lens         device, int32 [batch]
 * page_size        must be 64
 * request_status   device, uint32 [batch] (written)
 * checked_seq_lens device, int32 [batch] (written; may be the same buffer as
 *                  seq_lens only if no other work reads seq_lens concurrently)
 * Pointers need 4-byte alignment here. Tags are opaque 32-bit values.
 */
#define MLA_KV_CHECK_TAG_MISMATCH 0x1u
#define MLA_KV_CHECK_PAGE_RANGE 0x2u
#define MLA_KV_CHECK_BAD_LENGTH 0x4u
MLA_API mla_status mla_kv_check(const uint32_t* page_tags, int64_t num_pages,
                                const int32_t* block_table, const uint32_t* expected_tags,
                                int max_pages, const int32_t* seq_lens, int batch, int page_size,
                                uint32_t* request_status, int32_t* checked_seq_lens,
                                mla_stream_t stream);

/*
 * mla_decode_static_scratch -- mla_decode for callers that cannot allocate.
 *
 * No counterpart on the pages: this entry point exists for callers that may not
 * allocate device memory when they decode -- plug-ins inside an engine that has
 * reserved all device memory in its own pool and gives them no allocator, or
 * serving loops that forbid cudaMalloc (which can synchronise the device) after
 * start-up. It computes exactly what mla_decode computes, with the same kernels
 * and arguments, but takes no workspace: the split-KV scratch lives in one
 * array of MLA_STATIC_SCRATCH_BYTES inside this library's device image, held by
 * every GPU that loads the library until the process exits. It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *
 *  - Limit: returns MLA_ERR_WORKSPACE, enqueuing nothing, when the problem needs
 *    more scratch than MLA_STATIC_SCRATCH_BYTES, i.e. when
 *    mla_decode_workspace_size(batch, num_queries, num_heads, num_ctas) exceeds
 *    it: at 64 heads with one CTA per SM on a 152-SM GPU, batch x num_queries
 *    may be at most 229 rows.
 *  - Set-up: the first call on each device looks up the array's device address
 *    with that device current (cudaGetSymbolAddress). Make that first call
 *    before any stream capture. The address is kept per device ordinal and
 *    belongs to the runtime's primary context of that device: the entry point
 *    assumes that context for the whole process (no context of the caller's
 *    own, no cudaDeviceReset between calls).
 *  - Sharing: every call on a device uses the same array, which keeps the last
 *    call's contents. Calls that overlap on the GPU (for instance on two
 *    streams) race and give wrong results: order them on one stream or with
 *    events.
 *  - device_status: optional device pointer (may be NULL) that receives this
 *    call's MLA_DEVICE_ERR_* bits; the copy in the array is cleared afterwards,
 *    also when the call returns MLA_ERR_CUDA after some of its work was
 *    enqueued (the first error is returned).
 */
#define MLA_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
MLA_API mla_status mla_decode_static_scratch(const void* q, const void* kv_pages, int64_t num_pages,
                                             int page_size, int kv_dtype,
                                             const int32_t* block_table, int max_pages,
                                             const int32_t* seq_lens, int batch, int num_queries,
                                             int num_heads, float sm_scale, float kv_scale,
                                             int num_ctas, void* out, float* lse,
                                             unsigned* device_status, mla_stream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* PAGED_MLA_DECODE_MLA_H_ */
