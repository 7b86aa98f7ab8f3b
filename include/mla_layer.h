/*
 * mla_layer.h -- C ABI of the operators that feed the paged MLA decode
 * (mla_decode.h), in the same library (libmla_gb300.so): what an MLA layer's
 * attention runs between its hidden states and mla_decode_step, for one token
 * per request, for drafts and for prompt chunks.
 *
 *     mla_rms_norm             the layer's input norm (with the residual's
 *                              addition), the query latent's norm; output in
 *                              the input's type or in 8 bits with scales
 *     mla_rope                 rotary positions on part of each head
 *     mla_cache_append_tokens  many tokens per request into the paged latent
 *                              cache: latent norm, key rotation, quantisation
 *     mla_cache_gather         cached rows of any format back to dense bf16
 *
 * The path they serve: the fused projection q_a || kv_a_proj_with_mqa of the
 * hidden states ("vllm.models.glm5next.common.model", load_weights:
 * fused_qkv_a_proj) gives a query latent (q_lora_rank 768) and one row [c_kv
 * (512) || k_rope (64)] per token; both latents are normed, the query latent
 * is up-projected to heads of 192 + 64, the 64 are rotated to the token's
 * position, and the row is normed, rotated and cached (GLM-4.7-Flash record,
 * phantomic12 inference-research, configuration clause: q_lora_rank 768,
 * kv_lora_rank 512, qk_rope_head_dim 64, rope_theta 1000000).
 *
 * Conventions are mla_decode.h's: the caller owns every buffer, device
 * pointers are on the current device, calls are asynchronous on the given
 * stream, 0 is success, a negative MLA_ERR_* means that nothing was launched.
 * None of these calls needs a workspace, keeps state between calls, or reads
 * what it does not name: calls on separate buffers may overlap, and every
 * call can be captured in a CUDA graph.  Sums, scales and rotations are
 * computed in 32 bits and every output is rounded once.
 */
#ifndef MLA_LAYER_H_
#define MLA_LAYER_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define MLA_DTYPE_BF16 0
#define MLA_DTYPE_F16 1
#define MLA_DTYPE_F32 2

/* ------------------------------------------------------------------------
 * RMS norm
 * ------------------------------------------------------------------------ */
#define MLA_NORM_OUT_SAME 0        /* y in the input's type */
#define MLA_NORM_OUT_E4M3_E8M0 1   /* e4m3 with one e8m0 scale per 32 consecutive values */
#define MLA_NORM_OUT_E4M3_ROW 2    /* e4m3 with one f32 scale per row */

#define MLA_NORM_MAX_COLS 32768

typedef struct {
  int32_t rows;                /* >= 0 */
  int32_t cols;                /* 1 .. MLA_NORM_MAX_COLS */
  int32_t dtype;               /* MLA_DTYPE_*: x, residual, weight, residual_out and a
                                  MLA_NORM_OUT_SAME output */
  int32_t out_format;          /* MLA_NORM_OUT_* */
  float eps;                   /* >= 0, finite */
  int32_t reserved;            /* 0 */
  int64_t x_stride;            /* elements between rows, >= cols each */
  int64_t residual_stride;
  int64_t residual_out_stride;
  int64_t out_stride;
  int64_t scale_stride;        /* MLA_NORM_OUT_E4M3_E8M0: bytes between the scale rows,
                                  >= ceil(cols / 32); otherwise ignored */
} mla_norm_problem;

/*
 * mla_rms_norm -- for each row, in 32 bits,
 *
 *     h = x + residual                     (h = x without a residual)
 *     residual_out = h                     rounded once to dtype
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *
 * (The layer's input norm and the norms of the query and key-value latents:
 * GLM-4.7-Flash record, configuration clause, q_lora_rank and kv_lora_rank.)
 * y comes from the unrounded h, and is rounded once:
 *   MLA_NORM_OUT_SAME       out = y in dtype.
 *   MLA_NORM_OUT_E4M3_E8M0  the quantiser of the FP8 cache (mla_cache_append):
 *                           per 32 values e = ceil(log2(amax / 448)) clamped
 *                           to [-127, 127], scale byte e + 127, codes e4m3 of
 *                           y / 2^e to nearest even, saturating at 448; an
 *                           all-zero group gets scale byte 0 and zero codes.
 *                           The last group of a row may be shorter.  A NaN
 *                           stays a NaN code and does not enter amax.
 *   MLA_NORM_OUT_E4M3_ROW   scale = max(amax / 448, 2^-126) over the row, codes
 *                           e4m3 of y / scale to nearest even; y = code * scale.
 *                           A NaN anywhere in y makes the row's scale NaN.
 *
 *   x            : [rows][x_stride]
 *   residual     : NULL, or [rows][residual_stride]
 *   weight       : NULL (ones), or [cols].  Under an infinite one
 *                  MLA_NORM_OUT_E4M3_E8M0 gives a NaN code or +-448; the other
 *                  groups do not see it
 *   residual_out : NULL, or [rows][residual_out_stride]; needs residual.  May
 *                  be residual or x itself (same address and stride).
 *   out          : [rows][out_stride] of dtype or of bytes.  In dtype it may be
 *                  x, or the residual where residual_out is not, itself (same
 *                  address and stride).
 *   scales       : MLA_NORM_OUT_E4M3_E8M0: uint8 [rows][scale_stride];
 *                  MLA_NORM_OUT_E4M3_ROW: f32 [rows]; otherwise NULL
 * Pointers need the alignment of their elements; rows that start on 16-byte
 * boundaries are read and written in 16-byte pieces.  Elements behind a row's
 * cols are left as they were.  Finite rows of any size are normed, their
 * squares out of the 32-bit range too; a row with an infinity gives zeros (and
 * NaN for it), a row of zeros without an eps NaN.
 * Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT (a size, a missing or a surplus
 * pointer, an output that overlaps an input other than as said: rows of one
 * stride in bytes by their elements, as column ranges of one buffer, others by
 * their whole span), MLA_ERR_UNSUPPORTED (a dtype, an out_format, cols past the
 * limit), MLA_ERR_MISALIGNED or MLA_ERR_CUDA.
 */
MLA_API int mla_rms_norm(const mla_norm_problem* problem, const void* x, const void* residual,
                 const void* weight, void* residual_out, void* out, void* scales,
                 mla_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions
 * ------------------------------------------------------------------------ */
#define MLA_ROPE_INTERLEAVED 0   /* pair i is (x[2i], x[2i + 1]) */
#define MLA_ROPE_HALVES 1        /* pair i is (x[i], x[i + dim / 2]) */

#define MLA_ROPE_SCALING_NONE 0
#define MLA_ROPE_SCALING_LINEAR 1
#define MLA_ROPE_SCALING_PARTS 2
#define MLA_ROPE_SCALING_YARN 3

#define MLA_ROPE_MAX_DIM 256

/* How positions become angles.  Pair i of rope_dim / 2 turns by pos * g_i
 * radians, g_i from f_i = theta^(-2i / rope_dim):
 *   NONE    g_i = f_i.
 *   LINEAR  g_i = f_i / factor (positions interpolated).  Scaling theta itself
 *           (theta * factor^(rope_dim / (rope_dim - 2))) needs no mode: pass it.
 *   PARTS   by how often a pair turns over the original context, t_i =
 *           original_positions * f_i / (2 pi): w = (t_i - slow_rotations) /
 *           (fast_rotations - slow_rotations) clamped to [0, 1],
 *           g_i = w f_i + (1 - w) f_i / factor.
 *   YARN    the same blend on a ramp over the pair index: d(r) = rope_dim *
 *           ln(original_positions / (2 pi r)) / (2 ln theta), low =
 *           max(floor(d(fast_rotations)), 0), high = min(ceil(d(
 *           slow_rotations)), rope_dim - 1), w = 1 - clamp((i - low) /
 *           max(high - low, 0.001), 0, 1) (Peng et al., YaRN: Efficient
 *           Context Window Extension of Large Language Models, 2023).
 * The rotated values are multiplied by `amplitude`; 0 takes the scaling's
 * own: 0.1 ln(factor) + 1 for YARN (1 where factor <= 1), else 1. */
typedef struct {
  int32_t layout;              /* MLA_ROPE_INTERLEAVED or MLA_ROPE_HALVES */
  int32_t rope_dim;            /* even, 2 .. MLA_ROPE_MAX_DIM */
  int32_t scaling;             /* MLA_ROPE_SCALING_* */
  int32_t original_positions;  /* PARTS, YARN: context length before the extension, >= 1 */
  double theta;                /* > 1 */
  double factor;               /* > 0 */
  double fast_rotations;       /* PARTS, YARN: > slow_rotations > 0 (YaRN's beta 32 and 1) */
  double slow_rotations;
  double amplitude;            /* > 0, or 0 for the scaling's own */
} mla_rope_config;

/* Filled by mla_rope_make_plan; treat as opaque.  turns[i] is pair i's turn
 * per position in units of 2^-64 of a full turn: turns[i] * pos, wrapping,
 * is the angle's exact fraction of a turn, so far positions lose nothing.
 * (The frequencies are in 53 bits: an angle is off by less than pos * 2^-52
 * turns, and where a scaling's factor is below 1, which raises frequencies, by
 * less than pos * 2^-52 / factor.) */
typedef struct {
  mla_rope_config config;
  float amplitude;
  int32_t reserved;
  uint64_t turns[MLA_ROPE_MAX_DIM / 2];
} mla_rope_plan;

/* mla_rope_make_plan -- validate a configuration and compute its table (host
 * only, no CUDA call).  Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT or
 * MLA_ERR_UNSUPPORTED (a layout, scaling or rope_dim that is not listed). */
MLA_API int mla_rope_make_plan(const mla_rope_config* config, mla_rope_plan* plan_out);

typedef struct {
  int32_t tokens;              /* >= 0 */
  int32_t num_heads;           /* >= 1; num_heads * head_dim <= 2^25 - 1 */
  int32_t head_dim;            /* elements of a head, >= rope_offset + rope_dim */
  int32_t rope_offset;         /* first rotated element of a head */
  int32_t dtype;               /* MLA_DTYPE_* */
  int32_t transposed;          /* 1: turn by minus the angle (the transposed map: the
                                  gradient; with amplitude 1 also the inverse) */
  int64_t x_token_stride;      /* elements, 0 .. 2^31 - 1; out's heads must not overlap */
  int64_t x_head_stride;
  int64_t out_token_stride;
  int64_t out_head_stride;
} mla_rope_problem;

/*
 * mla_rope -- rotate elements [rope_offset, rope_offset + rope_dim) of every
 * head of token t to position positions[t] (the decode takes rotated queries:
 * GLM-4.7-Flash record, configuration clause, qk_rope_head_dim 64 of a 256
 * head).  The head's other elements are copied (nothing to do in place).
 *   x         : [tokens][num_heads][head_dim] by the strides
 *   positions : device int32 [tokens]; a negative one leaves that token's
 *               out as it was
 *   out       : as x; x itself with the same strides rotates in place
 * With pair (a, b) at angle t: a' = A (a cos t - b sin t), b' = A (a sin t +
 * b cos t), A the amplitude, in 32 bits, rounded once.
 * Returns MLA_OK, MLA_ERR_INVALID_ARGUMENT (a size or stride, a plan not made
 * by mla_rope_make_plan, an out that overlaps x otherwise: where their tokens'
 * or their heads' strides are equal the elements count, as in column ranges of
 * one buffer, else the whole span), MLA_ERR_UNSUPPORTED (a dtype, a stride or a
 * token's elements past the limits), MLA_ERR_MISALIGNED (less than the
 * elements' alignment) or MLA_ERR_CUDA.
 */
MLA_API int mla_rope(const mla_rope_problem* problem, const mla_rope_plan* plan, const void* x,
             const int32_t* positions, void* out, mla_stream_t stream);

/* ------------------------------------------------------------------------
 * The paged latent cache, many tokens at a time
 * ------------------------------------------------------------------------ */
/*
 * mla_cache_append_tokens -- write `tokens` rows into the paged latent cache:
 * prompt chunks, the drafts of a step, any mixture ("vllm.models.glm5next.
 * common.model", load_weights: the kv_a_proj_with_mqa output inside
 * fused_qkv_a_proj; GLM-4.7-Flash record, engine-kernel constraint (2): the
 * FP8 latent written with inlined scales).  Row t belongs to position
 * positions[t] of request requests[t]: page block_table[r][pos / P], slot
 * pos % P.  On the way the latent is normed (norm_weight given: c * weight /
 * sqrt(mean(c^2) + norm_eps), rows of any size as in mla_rms_norm) and the key
 * rotated to its position (rope given), in 32 bits, and the values rounded
 * once, to bf16 or by the cache's quantiser (the formulas of mla_cache_append;
 * without norm and rope the same bytes; a NaN becomes a NaN code in FP8 and a
 * NaN scale, byte 255, in FP4).
 *   problem     : the cache's shape as for mla_cache_append (batch = requests)
 *   rows        : bf16, token t's [c_kv (512) || k_rope (64)] at rows + t *
 *                 row_stride (elements, >= 576, a multiple of 8): a slice of a
 *                 wider projection needs no copy
 *   positions   : device int32 [tokens]; a negative one writes nothing
 *   requests    : device int32 [tokens], or NULL: token t is request t /
 *                 (tokens / batch), the same number of tokens for each
 *                 (tokens must be a multiple of batch)
 *   block_table : device int32 [batch][max_pages_per_seq]
 *   norm_weight : NULL, or bf16 [512]
 *   norm_eps    : >= 0, finite; read with norm_weight
 *   rope        : NULL, or a plan with rope_dim 64 (host)
 *   kv_cache    : written in place, in problem->kv_dtype's layout
 *   status      : nullable device uint32; a position past the request's pages
 *                 or a request outside [0, batch) sets MLA_STATUS_BAD_INDEX, a
 *                 page id outside [0, num_pages) MLA_STATUS_BAD_PAGE, and that
 *                 row is not written
 * Rows of one call must go to distinct slots.  Returns MLA_OK,
 * MLA_ERR_INVALID_ARGUMENT, MLA_ERR_MISALIGNED (rows, norm_weight or kv_cache
 * not on 16 bytes, a row_stride that is no multiple of 8), MLA_ERR_UNSUPPORTED
 * or MLA_ERR_CUDA.
 */
MLA_API int mla_cache_append_tokens(const mla_problem* problem, int32_t tokens, const void* rows,
                            int64_t row_stride, const int32_t* positions, const int32_t* requests,
                            const int32_t* block_table, const void* norm_weight, float norm_eps,
                            const mla_rope_plan* rope, void* kv_cache, uint32_t* status,
                            mla_stream_t stream);

/*
 * mla_cache_gather -- the cached rows of `tokens` (request, position) pairs as
 * dense bf16 rows [c_kv (512) || k_rope (64)]: the context of a chunked
 * prompt, whose keys and values are projected up from the latent, or a look
 * into a quantised cache (GLM-4.7-Flash record, engine-kernel constraint (2):
 * e4m3 or 4-bit latents with inlined e8m0 scales).  Values are code * 2^(scale -
 * 127), exact but for bf16's own range (scale byte 255 gives NaN).
 *   problem, positions, requests, block_table : as for mla_cache_append_tokens
 *   kv_cache : read, in problem->kv_dtype's layout
 *   out      : bf16, row t at out + t * out_stride (elements, >= 576, a
 *              multiple of 8).  A negative position leaves its row as it was;
 *              one that has no slot (bad request, position or page) is filled
 *              with zeros and reported in the status word.
 *   status   : nullable device uint32, bits as for mla_cache_append_tokens
 * out must not overlap the cache.  Returns as mla_cache_append_tokens.
 */
MLA_API int mla_cache_gather(const mla_problem* problem, int32_t tokens, const void* kv_cache,
                     const int32_t* positions, const int32_t* requests,
                     const int32_t* block_table, void* out, int64_t out_stride, uint32_t* status,
                     mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_LAYER_H_ */
