/*
 * skinny_window.h -- further operators around one decode window, on MI355X
 * (gfx950): the GEMV on 4-bit weights with group scales, a whole
 * mixture-of-experts layer, and log probabilities of given tokens.
 *
 * A window's step runs them one after another: the layer's rows go through
 * skinny_moe_run, the last layer's through a 4-bit output head
 * (skinny_w4_mm_run), its logits and the drafted tokens through
 * skinny_token_logprobs_run.
 *
 * Status codes, dtypes, memory, threading and errors are those of skinny.h:
 * every device pointer is the caller's, run calls allocate nothing, never
 * synchronise and only enqueue kernels on `stream`, so they can be captured
 * in a HIP graph; every argument is checked on the host before any HIP call,
 * and on an error nothing is enqueued.  Unless stated otherwise non-finite
 * inputs are outside the contract.
 */
#ifndef SKINNY_WINDOW_H
#define SKINNY_WINDOW_H

#include "skinny.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A workspace of these operators starts with arrival counters.  Only they have
 * to be zero before its first use: the first SKINNY_WINDOW_COUNTER_BYTES, or
 * nothing for a MoE layer whose router needs no workspace of its own
 * (skinny_mm_workspace_size of its plan for n = experts, k = d). */
#define SKINNY_WINDOW_COUNTER_BYTES 4096

/* --- 4-bit weights with group scales -------------------------------------- */

/* A 4-bit weight [n][k] in groups of `group` (32, 64 or 128) elements along k:
 *   weight (j, kk) = scale[j][kk/group] * (code(j, kk) - zero[j][kk/group])
 * as a real number: no weight is rounded to 16 bits (the block formats Q4_0
 * and Q2_0 above define theirs as rounded).
 *   codes   uint8 [n][k/2], two unsigned 4-bit codes per byte, element kk in
 *           byte kk/2, the low nibble for even kk; 16-byte aligned
 *   scales  [n][k/group] in the 16-bit type of the rows; 2-byte aligned
 *   zeros   uint8 [n][k/group], the zero points (0 .. 255; 0 .. 15 in use), or
 *           NULL: 8 everywhere */
typedef struct skinny_w4 {
  const void* codes;
  const void* scales;
  const void* zeros;
} skinny_w4;

/* C[0:m, 0:n] = A[0:m, :] . W for a decode window's rows and a 4-bit grouped
 * weight, in one launch that reads W once for all rows (past 2^27 columns, one
 * launch for each 2^27).  Products are exact
 * and summed in fp32, the group's scale is applied to its sum; row i of C at
 * any m equals the m = 1 call on that row bit for bit.
 *   A group's sum is the difference of sum (16 + code) a and (16 + zero) sum a,
 * so C is off by at most (group + k/group + 10) 2^-24 times the sum over k of
 * |scale| (32 + code + zero) |a|.  In root mean square that is 0.3 to 1.5 times
 * the error of an fp32 product of the same numbers (k = 2560; rows of mean 0,
 * of mean 4, and with one element of 1000).
 *   m        1 <= m <= SKINNY_GEMV_MAX_M
 *   n, k     1 <= n < 2^31; k a multiple of group, up to 2^24
 *   A        [m][lda] SKINNY_F16 or SKINNY_BF16 (a_dtype); lda >= k a multiple
 *            of 8 (0: k); 16-byte aligned
 *   C        [m][ldc] SKINNY_F32, SKINNY_F16 or SKINNY_BF16 (c_dtype, rounded to
 *            nearest even); ldc >= n (0: n); aligned to its element,
 *            overlapping no input (else SKINNY_ERR_INVALID_ARG)
 * All device pointers. */
SKINNY_API skinny_status skinny_w4_mm_run(int64_t m, int64_t n, int64_t k, int32_t group, const void* A,
                                          int64_t lda, int32_t a_dtype, const skinny_w4* W, void* C, int64_t ldc,
                                          int32_t c_dtype, void* stream);

/* --- A whole mixture-of-experts layer for a decode window ------------------ */

/* For each of m <= SKINNY_GEMV_MAX_M tokens x_t, with the router's weight
 * Wr [experts][d], experts of inner length `inter` and an optional shared
 * expert of inner length `shared_inter` behind a scalar gate:
 *   l_t   = Wr x_t                              fp32 logits
 *   S_t   = the topk largest of l_t (equal values by lower expert first)
 *   p_te  = exp(l_te) / sum of exp(l_t.) over S_t (SKINNY_MOE_RENORM) or over
 *           all experts
 *   f_e(x) = Wd_e (silu(Wg_e x) * (Wu_e x)),    silu(v) = v / (1 + e^-v)
 *   out_t = sum over e in S_t of p_te f_e(x_t)
 *           + sigmoid(wg . x_t) f_shared(x_t)   (when shared_inter > 0)
 * Products are summed in fp32; the inner values silu(.) * (.) are carried in 24
 * bits, the output rounded once (nearest even).  In an f16 layer with 16-bit
 * weights that holds for inner values from 2^-12 to 2^18 in magnitude: products
 * of smaller ones lose a bit for every power of two, larger ones become
 * infinite.  The distinct experts' weights are read once per window, an expert's
 * down weight once per 4 tokens that it serves.  A token's output is the same
 * bits at every m and beside any other tokens.
 *   struct_size   sizeof(skinny_moe_desc)
 *   dtype         SKINNY_F16 or SKINNY_BF16: x, the router, the gate's weight, the
 *                 scales, and the weights unless they are 4-bit
 *   w_dtype       the experts' and the shared expert's weights: dtype, or
 *                 SKINNY_W4 with groups of `group` (32, 64 or 128; else 0)
 *   out_dtype     SKINNY_F32, SKINNY_F16 or SKINNY_BF16
 *   max_m         1 .. SKINNY_GEMV_MAX_M
 *   d, inter, shared_inter   multiples of 32 (and of group), up to 2^20;
 *                 shared_inter 0: no shared expert.  Together with max_m, topk and
 *                 experts not so large that a launch would need more than 2^31
 *                 threads, 8 for each inner value of a window's experts and 16
 *                 for each of their outputs (else SKINNY_ERR_UNSUPPORTED)
 *   experts       topk .. SKINNY_MOE_MAX_EXPERTS; topk 1 .. SKINNY_TOPK_MAX
 *   ldx, ldo      row strides of x and out in elements, 0: d; ldx a multiple of 8
 *   flags         SKINNY_MOE_RENORM or 0
 *   num_cus       as in skinny_mm_desc */
#define SKINNY_MOE_RENORM 0x1u
#define SKINNY_MOE_MAX_EXPERTS 1024

typedef struct skinny_moe_desc {
  uint32_t struct_size;
  int32_t dtype;
  int32_t w_dtype;
  int32_t out_dtype;
  int32_t group;
  int32_t topk;
  int64_t max_m;
  int64_t d;
  int64_t inter;
  int64_t shared_inter;
  int64_t experts;
  int64_t ldx;
  int64_t ldo;
  uint32_t flags;
  int32_t num_cus;
} skinny_moe_desc;

/* Device pointers, 16-byte aligned (scales 2-byte; zeros any).  A 16-bit
 * weight is given in `codes`, with scales and zeros NULL; 4-bit weights come
 * with zero points all or none (else SKINNY_ERR_UNSUPPORTED).
 *   router       [experts][d]
 *   w13          [experts][2 inter][d]: expert e's gate rows, then its up rows
 *   w2           [experts][d][inter]
 *   shared13, shared2   [2 shared_inter][d], [d][shared_inter] (or all NULL)
 *   shared_gate  [d] (or NULL) */
typedef struct skinny_moe_weights {
  const void* router;
  skinny_w4 w13;
  skinny_w4 w2;
  skinny_w4 shared13;
  skinny_w4 shared2;
  const void* shared_gate;
} skinny_moe_weights;

typedef struct skinny_moe_plan skinny_moe_plan;

/* Validate `desc` and build a plan (host memory only, immutable). */
SKINNY_API skinny_status skinny_moe_plan_create(const skinny_moe_desc* desc, skinny_moe_plan** out_plan);
SKINNY_API void skinny_moe_plan_destroy(skinny_moe_plan* plan);

/* Bytes of device workspace every run of this plan needs: 16-byte aligned,
 * zero-filled (see SKINNY_WINDOW_COUNTER_BYTES) once before its first use; a
 * completed run leaves it ready for the next.  Two runs in flight at once must
 * not share one, and a graph that is replayed beside other runs needs its own.
 * A run is several launches: two host threads must not enqueue runs on one
 * workspace at once, not even on one stream. */
SKINNY_API skinny_status skinny_moe_workspace_size(const skinny_moe_plan* plan, size_t* bytes);

/* Enqueue the layer for m tokens (1 <= m <= max_m).
 *   x            [m][ldx], 16-byte aligned
 *   out          [m][ldo], aligned to its element, not overlapping x
 *   topk_idx     int32 [m][topk], topk_weight f32 [m][topk]: S_t and p_te, the
 *                largest logit first; 4-byte aligned; either may be NULL */
SKINNY_API skinny_status skinny_moe_run(const skinny_moe_plan* plan, int64_t m, const void* x,
                                        const skinny_moe_weights* weights, void* out, int32_t* topk_idx,
                                        float* topk_weight, void* workspace, size_t workspace_bytes, void* stream);

/* --- Log probabilities of given tokens ------------------------------------- */

/* For each row x of logits and its token t:
 *   logprob   f32 [m]  x_t - ln sum exp(x_j)
 *   entropy   f32 [m]  of the row's distribution, in nats
 *   rank      int32 [m]  1 + #{j : x_j > x_t, or x_j = x_t and j < t}
 *   top_ids   int32 [m][topk], top_logprobs f32 [m][topk]: the topk largest
 *             logits, equal values (IEEE ==) by lower index first, and their
 *             log probabilities
 * Sums are held in fp32.  A logit of -inf (masked out) has probability 0; a
 * row of nothing else gives log probabilities of -inf and an entropy of 0.  A
 * row that holds a NaN or +inf gives NaN (its ids lie in the row or are -1).
 * A token outside 0 .. vocab - 1 reads nothing: its logprob is NaN, its rank
 * 0, the row's other results are given.  For m <= SKINNY_GEMV_MAX_M a row's
 * results are the same bits at every m and wherever the row lies in memory.
 *   m, vocab     1 <= m, vocab <= 2^30, m * vocab <= 2^50
 *   logits       [m][ld] SKINNY_F32, SKINNY_F16 or SKINNY_BF16 (dtype), aligned to
 *                its element; ld >= vocab (0: vocab), any value
 *   tokens       [m] int32, or int64 when tokens64 is not 0; aligned to it
 *   topk         0 .. min(vocab, SKINNY_TOPK_MAX); 0: top_ids and top_logprobs are
 *                not written and may be NULL
 *   outputs      4-byte aligned, overlapping neither one another nor the inputs
 *   workspace    zero-initialised (see SKINNY_WINDOW_COUNTER_BYTES) device scratch of at least
 *                skinny_token_logprobs_workspace_size bytes, 16-byte aligned
 *                (may be NULL when that is 0); a completed run leaves it ready
 *                for the next, of any size it suffices for.  Two runs in
 *                flight at once must not share one.
 * All device pointers.  One launch (past 2^22 rows, one for each 2^22). */
SKINNY_API skinny_status skinny_token_logprobs_workspace_size(int64_t m, int64_t vocab, int32_t topk, size_t* bytes);
SKINNY_API skinny_status skinny_token_logprobs_run(int64_t m, int64_t vocab, const void* logits, int64_t ld,
                                                   int32_t dtype, const void* tokens, int32_t tokens64,
                                                   int32_t topk, float* logprob, float* entropy, int32_t* rank,
                                                   int32_t* top_ids, float* top_logprobs, void* workspace,
                                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SKINNY_WINDOW_H */
