/*
 * mla_chunk.h -- C ABI of the operators around a chunk of new tokens over the
 * paged latent cache (mla_decode.h), in the same library (libmla_gb300.so):
 *
 *     mla_chunk_attend    attention of any number of new tokens per request,
 *                         one to a whole prompt, over everything cached
 *     mla_cache_weights   the attention weight that queries give to each
 *                         cached row, added up
 *     mla_cache_evict     a request's cache cut to a budget of rows, those
 *                         with the greatest weights, without copying the rest
 *
 * The path they serve: a prompt is cached chunk by chunk (mla_layer.h,
 * mla_cache_append_tokens), each chunk attends to what is cached with it, the
 * queries of the prompt's end (or those of each decode step) leave weights
 * behind, and the rows that got least are evicted before decoding goes on over
 * the shorter cache (mla_decode_step).  The cached row is the latent shared by
 * all heads (GLM-4.7-Flash record, phantomic12 inference-research,
 * configuration clause: kv_lora_rank 512, qk_rope_head_dim 64), so a row has
 * one weight, the sum over heads, and keys carry their rotation, so rows may
 * stand in any slot.
 *
 * Conventions are mla_decode.h's: the caller owns every buffer, device
 * pointers are on the current device, calls are asynchronous on the given
 * stream, 0 is success, a negative MLA_ERR_* means that nothing was launched
 * or (MLA_ERR_CUDA) that a launch failed.  Nothing is kept between calls: a
 * workspace need not be cleared, and calls may overlap and be captured in CUDA
 * graphs as long as no two that overlap share a workspace or an output.
 */
#ifndef MLA_CHUNK_H_
#define MLA_CHUNK_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_CHUNK_MAX_HEADS 128
#define MLA_CHUNK_MAX_REQUESTS 8192

/* Filled by mla_chunk_make_plan; treat as opaque, keep it alive while in use. */
typedef struct {
  mla_problem problem;
  int32_t tokens;           /* query tokens of a call, all requests together */
  int32_t sm_count;
  int64_t context_tokens;   /* quantised caches: rows expanded at most */
  int32_t clusters;         /* pairs of CTAs that share the attention's work */
  int32_t mark;             /* set by mla_chunk_make_plan */
  int64_t ws_partial_o;     /* byte offset of f32 [2 * clusters][64][128][8]: columns in eights */
  int64_t ws_partial_lse;   /* byte offset of f32 [2 * clusters][128] */
  int64_t ws_segments;      /* byte offset of int32 [2 * clusters][4] */
  int64_t ws_starts;        /* byte offset of int32 [batch + 1][2]: a quantised cache's
                               requests in ws_rows */
  int64_t ws_rows;          /* byte offset of bf16 [context_tokens + 31 batch][576] */
  int64_t workspace_bytes;
} mla_chunk_plan;

/*
 * mla_chunk_make_plan -- validate a problem and lay out the workspace (host
 * only, no CUDA call).
 *   problem        : the cache and the queries: batch (up to
 *                    MLA_CHUNK_MAX_REQUESTS), num_heads (1 .. MLA_CHUNK_MAX_HEADS), page_size,
 *                    num_pages, max_pages_per_seq, kv_dtype, causal, sm_scale and the
 *                    widths of the row; q_len is not read, topk_width must be 0
 *   tokens         : query tokens of all requests together, >= 0
 *   context_tokens : quantised caches: the most rows that the requests of one
 *                    call have cached together, a page that several share counted
 *                    for each of them (their rows are expanded to
 *                    bf16 in the workspace, 1,152 bytes each and up to 31 rows
 *                    more a request); MLA_KV_BF16: not read
 *   sm_count       : streaming multiprocessors to fill (152 on GB300), > 0
 * Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT or MLA_ERR_UNSUPPORTED.
 */
MLA_API int mla_chunk_make_plan(const mla_problem* problem, int32_t tokens, int64_t context_tokens,
                                int32_t sm_count, mla_chunk_plan* plan_out,
                                size_t* workspace_bytes);

/*
 * mla_chunk_attend -- causal attention of new tokens over the paged cache, in
 * latent space (GLM-4.7-Flash record, the MLA decode kernel class: absorbed
 * queries against the shared latent plus the decoupled RoPE key; the chunk of
 * a prompt takes the same form).  Request b's new tokens are query_starts[b]
 * .. query_starts[b + 1] - 1, n_b of them, any number from none on; its T_b =
 * seq_lens[b] cached rows include theirs.  Token j of the request (from 0)
 * sees the first T_b - n_b + j + 1 rows (all T_b where problem.causal is 0).
 * For each of its heads
 *     s_t = sm_scale q_hat . row_t     lse = ln sum_t exp(s_t)
 *     o   = sum_t exp(s_t - lse) c_kv[t]
 * with scores, sums and accumulation in 32 bits; the weights are rounded to
 * bf16 for the product with the rows, relative to a running maximum, and o is
 * divided by the sum of the rounded ones.  A row that sees nothing gets o = 0
 * and lse = -inf.
 *   q_hat        : bf16 [tokens][num_heads][576], absorbed (mla_q_absorb)
 *   query_starts : device int32 [batch + 1], not descending, from 0 on and at
 *                  most tokens (values outside are taken as the nearest bound
 *                  and reported); tokens from query_starts[batch] on are padding
 *   kv_cache, block_table, seq_lens : as for mla_decode_run, cached rows of
 *                  every kv_dtype.  Slots that hold no row of the request
 *                  (behind its last) may hold anything, NaN too; a row of the
 *                  request that holds a NaN or an infinity may also reach tokens
 *                  of its call that do not see it (their weight for it is 0)
 *   workspace    : device buffer of workspace_bytes >= plan->workspace_bytes
 *   o_lat        : bf16 [tokens][num_heads][512] (the decode's is f32; a chunk's
 *                  goes into a matrix product of its own); padding is left as it was
 *   lse          : f32 [tokens][num_heads]; padding is left as it was
 *   status       : nullable device uint32; MLA_STATUS_BAD_PAGE: a block-table entry
 *                  outside [0, num_pages), whose rows are masked out;
 *                  MLA_STATUS_BAD_INDEX: a query start or length out of range, or
 *                  more rows than context_tokens, the surplus masked out;
 *                  MLA_STATUS_TIMEOUT: an internal wait hit its limit
 * The workspace and each output share no memory with an input or one another
 * (MLA_ERR_INVALID_ARGUMENT).
 * Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT, MLA_ERR_MISALIGNED (a pointer not on
 * 16 bytes; o_lat: 32; int32, lse and status: 4), MLA_ERR_WORKSPACE_TOO_SMALL or
 * MLA_ERR_CUDA.
 */
MLA_API int mla_chunk_attend(const mla_chunk_plan* plan, const void* q_hat,
                             const int32_t* query_starts, const void* kv_cache,
                             const int32_t* block_table, const int32_t* seq_lens, void* workspace,
                             size_t workspace_bytes, void* o_lat, float* lse, uint32_t* status,
                             mla_stream_t stream);

/*
 * mla_cache_weights -- how much of their attention queries give to each cached
 * row, added to what earlier ones gave:
 *     weights_out[b][t] = weights_in[b][t] + sum over the request's new tokens
 *                         that see row t, and their heads, of exp(s_t - lse)
 * for t < T_b; entries from T_b on are left as they were.  The queries may be
 * those of a decode step, of a chunk, or the last tokens of one (their rows of
 * q_hat and lse, query_starts over them alone: causality counts from the end of
 * the cache).  A query whose lse is -inf (it saw nothing) gives nothing.  The
 * sum has a fixed order: equal calls give equal bits.
 *   lse         : f32 [tokens][num_heads], from mla_chunk_attend or mla_decode_step
 *   weights_in  : f32 [batch][stride], or NULL for zeros
 *   weights_out : f32 [batch][stride]; may be weights_in
 *   stride      : elements between two requests' weights, >= 1; slots from stride
 *                 on are neither read nor written
 * The other arguments and the result are mla_chunk_attend's (weights: 4-byte
 * alignment; weights_out may only be weights_in itself, not overlap it).
 */
MLA_API int mla_cache_weights(const mla_chunk_plan* plan, const void* q_hat, const float* lse,
                              const int32_t* query_starts, const void* kv_cache,
                              const int32_t* block_table, const int32_t* seq_lens, void* workspace,
                              size_t workspace_bytes, const float* weights_in, float* weights_out,
                              int64_t stride, uint32_t* status, mla_stream_t stream);

/* Filled by mla_evict_make_plan; treat as opaque. */
typedef struct {
  mla_problem problem;
  int32_t budget, sinks, recent;
  int32_t mark;             /* set by mla_evict_make_plan */
  int64_t most_moves;       /* rows that one request's eviction can move */
  int64_t ws_counts;        /* byte offset of int32 [batch] */
  int64_t ws_moves;         /* byte offset of int32 [batch][most_moves][2] */
  int64_t workspace_bytes;
} mla_evict_plan;

/*
 * mla_evict_make_plan -- validate an eviction and lay out its workspace (host
 * only, no CUDA call).
 *   problem : the cache: batch (up to MLA_CHUNK_MAX_REQUESTS), page_size, num_pages,
 *             max_pages_per_seq, kv_dtype and the widths of the row; the other
 *             fields are not read
 *   budget  : rows that each request keeps at most, >= 1
 *   sinks   : tokens of positions below this are kept before all others, >= 0
 *   recent  : so are the tokens of the last `recent` positions, >= 0
 * An eviction's launches are sized for 152 multiprocessors (GB300).
 * Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT or MLA_ERR_UNSUPPORTED.
 */
MLA_API int mla_evict_make_plan(const mla_problem* problem, int32_t budget, int32_t sinks,
                                int32_t recent, mla_evict_plan* plan_out, size_t* workspace_bytes);

/*
 * mla_cache_evict -- cut each request's cache to the plan's budget.  A request
 * of T rows, T above the budget, keeps `budget` of them: first those whose
 * position is below `sinks` or above (its highest position - `recent`), then
 * those with the greatest weights; of equal ones those in the lowest slots (a
 * NaN counts as less than every number, -0 as 0).  A row that is kept and
 * stands in a slot below the budget stays there.  The others, in the order of
 * their slots, move into the slots below the budget that became free, in the
 * order of those, with their weights and positions; attention does not depend
 * on the order of rows, and `positions` says which token each slot holds.
 * Requests of at most `budget` rows stay as they are.
 *   kv_cache      : rows are moved in place, in problem.kv_dtype's layout
 *   block_table   : int32 [batch][max_pages_per_seq]; not changed (pages from
 *                   ceil(budget / page_size) on hold nothing any more)
 *   seq_lens      : device int32 [batch], T_b
 *   weights       : f32 [batch][stride], of the slots (mla_cache_weights)
 *   positions     : int32 [batch][stride], the slots' tokens, >= 0
 *   stride        : elements between two requests' entries, >= 1; lengths above it
 *                   are taken as it and reported
 *   seq_lens_out  : int32 [batch]: min(T_b, budget)
 *   weights_out   : f32 [batch][stride]: the kept rows' weights, 0 for the slots
 *                   given up (budget .. T_b - 1), as it was from T_b on
 *   positions_out : int32 [batch][stride]: the kept rows' positions, -1 for the
 *                   slots given up, as it was from T_b on
 *                   Each output may be its input itself, and overlaps nothing else.
 *   status        : nullable device uint32; MLA_STATUS_BAD_PAGE: a row could not be
 *                   moved, its page or its new one being outside [0, num_pages);
 *                   MLA_STATUS_BAD_INDEX: a length out of range, taken as the
 *                   nearest bound
 * Requests must not share the pages that rows are moved in.  Returns MLA_OK,
 * MLA_ERR_INVALID_ARGUMENT, MLA_ERR_MISALIGNED (kv_cache and workspace 16 bytes,
 * the others 4), MLA_ERR_WORKSPACE_TOO_SMALL or MLA_ERR_CUDA.
 */
MLA_API int mla_cache_evict(const mla_evict_plan* plan, void* kv_cache, const int32_t* block_table,
                            const int32_t* seq_lens, const float* weights,
                            const int32_t* positions, int64_t stride, void* workspace,
                            size_t workspace_bytes, int32_t* seq_lens_out, float* weights_out,
                            int32_t* positions_out, uint32_t* status, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CHUNK_H_ */
