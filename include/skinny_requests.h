/*
 * skinny_requests.h -- operators around the projections of a decode step that
 * serves several requests at once, on MI355X (gfx950): the residual's addition
 * with a root-mean-square norm, low-rank adapters beside a shared projection,
 * and penalties, biases and grammar masks on logits.
 *
 * A step runs them one after another: skinny_rms_norm_run gives a layer's rows,
 * a projection (skinny_mm_run, skinny_w4_mm_run) multiplies them by the shared
 * weight and skinny_adapters_run adds each request's own part; after the head,
 * skinny_adjust_logits_run prepares the logits for skinny_token_logprobs_run or
 * a sampler.
 *
 * Status codes, dtypes, memory, threading and errors are those of skinny.h:
 * every device pointer is the caller's, run calls allocate nothing, never
 * synchronise and only enqueue kernels on `stream`, so they can be captured
 * in a HIP graph; every argument is checked on the host before any HIP call,
 * and on an error nothing is enqueued.  Unless stated otherwise non-finite
 * inputs are outside the contract.  A row stride of 0 means dense rows; strides go
 * up to 2^40 elements, and rows times stride up to 2^60.
 */
#ifndef SKINNY_REQUESTS_H
#define SKINNY_REQUESTS_H

#include "skinny.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --- The residual's addition and a root-mean-square norm -------------------- */

/* For each row x of m rows of d values, with the residual r (or 0 without one):
 *   h            = x + r                                    in fp32
 *   residual_out = h, rounded to the residual's type
 *   y            = h * weight / sqrt(mean(h^2) + eps)       in fp32
 *   out          = y, rounded to its type (nearest even)
 *   scales_g     = max(max |y_j| over group g / 448, 2^-126)
 *   q_j          = y_j / scales_g in fp32, rounded to 8 bits (e4m3, nearest even):
 *                  q_j * scales_g stands for y_j
 * The norm is that of the unrounded sum h, and q is rounded from the unrounded y.
 * Groups are `group` (32, 64 or 128) consecutive columns, the row's last one
 * what is left, or the whole row (group 0).  A row's results do not depend on
 * the other rows: they are the same bits at every m.  mean(h^2) is held in
 * fp32: rows whose sum of squares overflows it (|h| near 2^63) come out as 0.
 * A NaN or infinity stays in its row.  The 8-bit output is for an 8-bit product of
 * the caller's own: this library's products take 16-bit rows and block formats.
 *   m, d          1 <= m <= 2^31, 1 <= d <= 2^24
 *   x             [m][ldx] SKINNY_F32, SKINNY_F16 or SKINNY_BF16 (x_dtype)
 *   residual      [m][ldr] of any of these types (r_dtype), or NULL
 *   weight        [d] of any of them (w_dtype), or NULL: 1 everywhere
 *   eps           >= 0, finite; with eps = 0 a row of zeros gives NaN, and rows of
 *                 |h| below 2^-63 lose bits of their squares
 *   residual_out  [m][ldro] of r_dtype, or NULL; may be `residual` itself (the
 *                 same rows), not given without a residual
 *   out           [m][ldo] SKINNY_F32, SKINNY_F16 or SKINNY_BF16 (out_dtype), or
 *                 NULL; may be x itself (the same rows and type)
 *   q, scales     uint8 [m][ldq] and f32 [m][groups], dense; both or neither
 *   At least one of residual_out, out and q.  Rows and vectors are aligned to
 *   their element, strides are any from the rows' length on; beyond what is
 *   allowed above, outputs overlap neither one another nor an input, each
 *   counted from its first element to its last (else SKINNY_ERR_INVALID_ARG).
 * All device pointers.  One launch (past 2^30 threads, several). */
SKINNY_API skinny_status skinny_rms_norm_run(int64_t m, int64_t d, const void* x, int64_t ldx, int32_t x_dtype,
                                             const void* residual, int64_t ldr, int32_t r_dtype, const void* weight,
                                             int32_t w_dtype, float eps, void* residual_out, int64_t ldro, void* out,
                                             int64_t ldo, int32_t out_dtype, void* q, int64_t ldq, float* scales,
                                             int32_t group, void* stream);

/* --- Low-rank adapters beside a shared projection --------------------------- */

/* A pool of adapters for one projection [n][k], in device memory:
 *   A        [count][rank][k] of dtype (SKINNY_F16 or SKINNY_BF16)
 *   B        [count][n][rank] of dtype
 *   ranks    int32 [count], each adapter's own rank (at most `rank`), or NULL:
 *            rank.  What A and B hold past it is not used and may be anything.
 *            A rank outside 1 .. rank counts as 0: the adapter adds nothing.
 *   scaling  f32 [count], or NULL: 1
 *   count    1 .. SKINNY_ADAPTERS_MAX
 *   rank     a multiple of 8, up to SKINNY_ADAPTER_RANK_MAX
 *   k, n     k a multiple of 8, up to 2^24; 1 <= n <= 2^24
 * A and B are 16-byte aligned, ranks and scaling 4-byte. */
#define SKINNY_ADAPTERS_MAX 8192
#define SKINNY_ADAPTER_RANK_MAX 256

typedef struct skinny_adapters {
  uint32_t struct_size; /* sizeof(skinny_adapters) */
  int32_t dtype;
  int64_t count, rank, k, n;
  const void* A;
  const void* B;
  const int32_t* ranks;
  const float* scaling;
} skinny_adapters;

/* For each of m rows x_t whose request uses adapter a = ids[t]:
 *   out_t = base_t + scaling[a] * B[a] (A[a] x_t)
 * and out_t = base_t where ids[t] lies outside 0 .. count - 1 (no adapter; its x
 * is not read).  `base` is the shared projection's output, or NULL: 0.  Sums are
 * held in fp32, the inner values A x are carried in 24 bits, and the output is
 * rounded once.  Rows of one adapter are multiplied together wherever they
 * stand: 16 of them share a read of its weights; past 256 rows 64 share one of A, and
 * 64 one of B where tiles are many and ranks short (else 16).  A row's results do
 * not depend on the other rows' values; for m <= SKINNY_GEMV_MAX_M they are the same
 * bits at every m.
 *   m          1 <= m <= 2^20
 *   x          [m][ldx] of the adapters' dtype; ldx a multiple of 8; 16-byte
 *              aligned
 *   ids        int32 [m], or int64 when ids64 is not 0; aligned to it
 *   base       [m][ldb] SKINNY_F32 or the adapters' dtype (base_dtype), aligned to
 *              its element
 *   out        [m][ldo] SKINNY_F32 or the adapters' dtype (out_dtype), aligned to
 *              its element; may be base itself (the same rows and type), and
 *              overlaps nothing else
 *   workspace  device scratch of at least skinny_adapters_workspace_size bytes,
 *              16-byte aligned, of any contents, apart from every operand.  Two runs
 *              in flight at once must not share one; a run is up to three launches
 *              over it, so two host threads must not enqueue runs on one workspace
 *              at once. */
SKINNY_API skinny_status skinny_adapters_workspace_size(const skinny_adapters* adapters, int64_t m, size_t* bytes);
SKINNY_API skinny_status skinny_adapters_run(const skinny_adapters* adapters, int64_t m, const void* x, int64_t ldx,
                                             const void* ids, int32_t ids64, const void* base, int64_t ldb,
                                             int32_t base_dtype, void* out, int64_t ldo, int32_t out_dtype,
                                             void* workspace, size_t workspace_bytes, void* stream);

/* --- Penalties, biases and grammar masks on logits --------------------------- */

/* What changes a row's logits.  Every pointer may be NULL.
 *   history         [m][ldh] the rows' token ids so far, int32, or int64 when
 *                   tokens64 is not 0; room for history_len each.  Ids outside
 *                   0 .. vocab - 1 do not count.
 *   lengths         int32 [m], how many of them a row has (NULL: history_len)
 *   prompt_lengths  int32 [m], how many of those, from the first on, are the
 *                   prompt's (NULL: 0); the others were generated
 *   repetition      f32 [m], theta > 0 (NULL: 1)
 *   frequency       f32 [m] (NULL: 0)
 *   presence        f32 [m] (NULL: 0)
 *   bias_ids        [m][biases] token ids like the history's, dense; ids outside
 *                   0 .. vocab - 1 fill a list up
 *   bias_values     f32 [m][biases], dense
 *   mask            int32 [masks][ldm], bit j % 32 of word j / 32 set where token j
 *                   is allowed
 *   mask_rows       int32 [m], the mask of each row, outside 0 .. masks - 1: none
 *                   (NULL: row i has mask i, and masks >= m)
 * Lengths are taken as 0 .. history_len, prompt_lengths as 0 .. the row's length. */
typedef struct skinny_logit_rules {
  uint32_t struct_size; /* sizeof(skinny_logit_rules) */
  int32_t tokens64;
  const void* history;
  int64_t ldh, history_len;
  const int32_t* lengths;
  const int32_t* prompt_lengths;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const void* bias_ids;
  const float* bias_values;
  int64_t biases;
  const int32_t* mask;
  int64_t ldm, masks;
  const int32_t* mask_rows;
} skinny_logit_rules;

/* For each row and each token j, in fp32 and in this order, with c_j the times j
 * was generated and s_j whether it occurs in prompt or generated tokens at all:
 *   x_j = s_j ? (x_j > 0 ? x_j / theta : x_j * theta) : x_j
 *   x_j = x_j - (frequency * c_j + presence * [c_j > 0])
 *   x_j = x_j + the biases listed for j, added up in the list's order
 *   x_j = -inf where the row's mask does not allow j
 * rounded once to the output's type.  Logits of -inf stay (theta > 0); a NaN
 * stays unless it is masked.  A row whose mask allows nothing is -inf
 * throughout.  Results do not depend on the order in which anything runs.
 *   m, vocab     1 <= m, vocab <= 2^30, m * vocab <= 2^50
 *   logits       [m][ld] SKINNY_F32, SKINNY_F16 or SKINNY_BF16 (dtype)
 *   out          [m][ldo] SKINNY_F32 or the logits' dtype (out_dtype).  May be the
 *                logits themselves (the same rows and type): then only the
 *                logits that change are written.  Else it overlaps no input.
 *   history_len  0 .. 2^24; biases 0 .. 2^16
 *   Everything is aligned to its element; strides are any from the rows' length on
 *   (ldm from ceil(vocab / 32) on).
 * All device pointers.  One launch (past 2^30 threads, several). */
SKINNY_API skinny_status skinny_adjust_logits_run(int64_t m, int64_t vocab, const void* logits, int64_t ld,
                                                  int32_t dtype, const skinny_logit_rules* rules, void* out,
                                                  int64_t ldo, int32_t out_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_REQUESTS_H */
