/*
 * moe_ops.h -- C ABI of the FP8 layer operators: the operators around and
 * inside a routed MoE layer whose weights are e4m3 with one scale per block
 * of 128 x 128, for any number of token rows (one decoded token to prompts
 * of thousands), and the other operators of a decoding step: the paged cache
 * of keys and values, attention over it, and the verification of drafted
 * tokens.  They are in the same library as moe_router.h and follow its
 * conventions: device pointers, the caller's memory and stream, every check
 * on the host before the first launch, moe_status with moe_last_error(), no
 * allocation and no synchronisation (moeop_read_device_status excepted), and
 * capture into CUDA graphs.  The first product on a device looks up what the
 * library keeps per device: make that call before a capture.
 *
 * FP8 rows [T][K]: e4m3 (bias 7, no infinity) codes, row-major, and fp32
 * scales [T][ceil(K/128)]; value = code * scale of its 128 inputs.
 * FP8 weights [N][K]: e4m3 codes, row-major, and fp32 scales
 * [ceil(N/128)][ceil(K/128)]; value = code * scale of its 128 x 128 block.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_router.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOEOP_BLOCK 128            /* inputs (and outputs) that share a scale */
#define MOEOP_MAX_NORM_HIDDEN 32768
#define MOEOP_MAX_EXPERTS 1024
#define MOEOP_MAX_TOPK 64
#define MOEOP_MAX_GROUPS 32

enum { MOEOP_BF16 = 0, MOEOP_FP16 = 1, MOEOP_FP32 = 2 };
enum { MOEOP_E4M3 = 3 };           /* of a cache only */
enum { MOEOP_GROUP_MAX = 0, MOEOP_GROUP_TOP2 = 1 };

/* Root-mean-square norm with the residual's addition and an FP8 output.
 *   s = x (+ residual);  y = s / sqrt(mean(s^2) + eps) * weight
 * in fp32, from the unrounded sum.  x, residual, weight, y and residual_out
 * have type `dtype`; x and residual have row strides in elements.  Each of
 * y, residual_out and (q, scales) is optional (NULL), one of y and q must be
 * given.  residual_out receives s and may be x or residual itself (the same
 * pointer and row stride: residual_out is contiguous, so the stride is then
 * hidden).  q, scales: FP8 rows of the unrounded y; scale =
 * max(largest magnitude of the 128, 1e-30) / 448.
 * hidden: 1..32768, any; the last 128 may be partial. */
MOE_API moe_status moeop_rms_norm(const void *x, int64_t x_stride, const void *residual,
                                  int64_t residual_stride, const void *weight, int rows,
                                  int hidden, int dtype, float eps, void *y, void *residual_out,
                                  uint8_t *q, float *scales, void *stream);

/* Routing of `rows` token rows to experts.
 *   p = softmax(logits) or sigmoid(logits); key = p + bias, or the logit
 *   itself without a bias (both scorings increase with it).
 * The experts are `groups` contiguous groups of equal size; a group scores
 * the largest p + bias of its experts, or the sum of its two largest
 * (MOEOP_GROUP_TOP2); the best group_limit groups stay, and the top_k largest
 * keys in them are taken, in descending order.  Ties (of groups and of
 * experts) go to the lower index.  Which key is larger is decided as if
 * everything were computed in 64 bits.
 * wts: p of the chosen (never the bias), divided by their sum with
 * norm_topk_prob, times routed_scaling_factor.
 * A logit of -inf or NaN takes its expert out of the row, a bias of -inf or
 * NaN out of all rows: it is not taken and counts for no group.  (The softmax
 * goes over all logits that are not -inf or NaN, whatever the biases; +inf is
 * no logit, its softmax has NaN weights.)  A bias of +inf puts its expert, and
 * its group, before all others; its weight is p as ever.  Slots for which no
 * expert is left get id -1 and weight 0. */
typedef struct moeop_route_config {
    int num_experts;             /* 1..1024 */
    int top_k;                   /* 1..min(64, group_limit * num_experts / groups) */
    int scoring;                 /* MOE_SCORING_SOFTMAX or _SIGMOID */
    int groups;                  /* 1..32, divides num_experts */
    int group_limit;             /* 1..groups */
    int group_score;             /* MOEOP_GROUP_MAX or _TOP2 */
    int norm_topk_prob;          /* 0 or 1 */
    float routed_scaling_factor;
    int dtype;                   /* of the logits */
} moeop_route_config;

MOE_API moe_status moeop_route_topk(const moeop_route_config *cfg, const void *logits,
                                    int64_t logits_stride, const float *bias, int rows,
                                    int32_t *ids, float *wts, void *stream);

/* out[m][n] = sum_k A[m][k] B[n][k], A FP8 rows [m][k] (row stride a_stride
 * bytes), B FP8 weights [n][k] (row stride b_stride bytes), out of type
 * out_dtype, contiguous.  The products of 128 inputs are summed on the
 * tensor cores in fp32, scaled and added in fp32, and rounded once.
 * k and both strides: multiples of 16; a and b 16-byte aligned. */
MOE_API moe_status moeop_matmul_fp8(const uint8_t *a, int64_t a_stride, const float *a_scales,
                                    const uint8_t *b, int64_t b_stride, const float *b_scales,
                                    int m, int n, int k, void *out, int out_dtype, void *stream);

/* The routed experts of `rows` FP8 rows q [rows][hidden]:
 *   g, u = q . gate[e]^T, q . up[e]^T;  h = silu(g) * u, held as FP8 rows;
 *   out[t] = sum_j wts[t][j] * (h . down[e]^T)  (+ addend[t]), e = ids[t][j]
 * in slot order.  An id outside [0, num_experts) contributes nothing.  The
 * products of the down projection are held in fp32 until they are weighted and
 * added, in fp32; out is rounded once.  addend (bf16, may be NULL) and out
 * (bf16) are contiguous; out may be addend.  All weights of a kind are one
 * stack: gate, up [E][inter][hidden], down [E][hidden][inter], each with its
 * scales [E][..][..].  A dense FP8 MLP is the case num_experts = top_k = 1. */
typedef struct moeop_experts_config {
    int hidden;                  /* multiple of 128, 128..32768 */
    int inter;                   /* multiple of 128, 128..32768 */
    int num_experts;             /* 1..1024 */
    int top_k;                   /* 1..64 */
} moeop_experts_config;

typedef struct moeop_experts_weights {
    const uint8_t *gate, *up, *down;
    const float *gate_scales, *up_scales, *down_scales;
} moeop_experts_weights;

/* Bytes of workspace for calls of up to `rows` rows (0 = refused). */
MOE_API size_t moeop_experts_workspace_size(const moeop_experts_config *cfg, int rows);

/* ws: 256-byte aligned device memory, needs no initialisation; calls that
 * overlap on the GPU need one each. */
MOE_API moe_status moeop_experts_fp8(const moeop_experts_config *cfg,
                                     const moeop_experts_weights *w, const uint8_t *q,
                                     const float *scales, const int32_t *ids, const float *wts,
                                     const uint16_t *addend, uint16_t *out, int rows, void *ws,
                                     size_t ws_bytes, void *stream);

/* A paged cache of keys and values.  Page p, key/value head h, place i of the
 * page: dim elements at k + p * k_stride + (h * page + i) * dim, so that a head's
 * places of a page are one contiguous run.  e4m3: codes, and an fp32 scale for
 * each head and place (k_scales + p * k_scales_stride + h * page + i); value =
 * code * scale.  A slot is a place in the cache: page number * page + i.  The
 * strides are in elements, from one page to the next.
 * All four arrays and their strides 16-byte aligned; scales NULL unless e4m3. */
typedef struct moeop_kv_cache {
    void *k, *v;
    float *k_scales, *v_scales;
    int64_t k_stride, v_stride, k_scales_stride, v_scales_stride;
    int pages, heads;            /* pages * page < 2^31; heads 1..1024 */
    int page;                    /* a multiple of 16, 16..1024 */
    int dim;                     /* 64, 128 or 256 */
    int type;                    /* MOEOP_BF16, MOEOP_FP16 or MOEOP_E4M3 */
} moeop_kv_cache;

/* Write the keys and values of `tokens` tokens, [tokens][heads][dim] with row
 * strides in elements, to their slots.  e4m3: scale = max(largest magnitude of
 * the dim, 1e-30) / 448, code = e4m3(value / scale), from any dtype (a NaN is
 * the code of NaN and leaves the scale to the others; an infinity makes all of
 * its row NaN); a cache of 16 bits takes rows of its own type and keeps them as
 * they are.  A slot outside the cache is passed over.  The slots of a call are
 * distinct: what a slot given twice holds afterwards is not defined (the others
 * are not touched by it).  k, v and their strides 16-byte aligned. */
MOE_API moe_status moeop_kv_write(const moeop_kv_cache *cache, const void *k, int64_t k_stride,
                                  const void *v, int64_t v_stride, int dtype,
                                  const int32_t *slots, int tokens, void *stream);

/* Read slots back: k, v [tokens][heads][dim] of type dtype, contiguous, 16-byte
 * aligned.  A slot outside the cache gives zeros. */
MOE_API moe_status moeop_kv_read(const moeop_kv_cache *cache, const int32_t *slots, int tokens,
                                 void *k, void *v, int dtype, void *stream);

/* Attention of the last `rows` tokens of each of `batch` sequences over their
 * cached tokens (their own among them: write first).  Sequence b has lengths[b]
 * tokens (negative: none; more than width * page: that many); token j is at
 * place j % page of page table[b][j / page], row r at position
 * lengths[b] - rows + r.  A row sees the tokens up to its own position, with a
 * window only the last `window` of them, its own included; a page number
 * outside the cache takes its tokens out.
 *   out = sum_j softmax(scale * q . k_j)_j v_j
 * with each of the group = q_heads / heads query heads of a key/value head.  A
 * row that sees nothing (a position before the first token, length 0), or only
 * scores of -inf, is zero.  What a row does not see does not reach it, NaN and
 * infinities included.
 * q [batch][rows][q_heads][dim] with strides (elements) of batch and rows, out the
 * same, contiguous, both of type dtype: bf16 or fp16, the cache's own type where
 * that is one of 16 bits.  Products, softmax statistics and sums are in fp32;
 * probabilities enter the second product as two 16-bit numbers whose sum is
 * within 2^-16 of them (bf16), or within 2^-22 of them or 2^-44 of the row's
 * largest (fp16; e4m3: of the probability times the value's scale).  out is
 * rounded once.
 * Scores beyond the range of fp32 give NaN, as they do in a softmax; an infinite
 * value that a row sees gives an infinity or NaN.
 * The first call on a device looks up what the library keeps per device. */
typedef struct moeop_attend_config {
    int batch;                   /* 0..2048 */
    int rows;                    /* 1..64 */
    int q_heads;                 /* a multiple of the cache's heads; rows * group <= 256 */
    int width;                   /* pages in a row of the table, >= 1 */
    int window;                  /* 0 = none */
    float scale;                 /* below 2^127 in magnitude */
    int dtype;                   /* of q and out */
} moeop_attend_config;

/* Bytes of workspace for calls of this batch (and smaller ones), rows, q_heads,
 * heads and dim (0 = refused).  It is initialised once, by
 * moeop_attend_workspace_init, and every call leaves it ready for the next, of
 * the same or another shape.  256-byte aligned; calls that overlap on the GPU
 * need one each. */
MOE_API size_t moeop_attend_workspace_size(int batch, int rows, int q_heads, int heads, int dim);
MOE_API moe_status moeop_attend_workspace_init(void *ws, size_t ws_bytes, void *stream);
MOE_API moe_status moeop_attend_paged(const moeop_attend_config *cfg, const moeop_kv_cache *cache,
                                      const void *q, int64_t q_batch_stride, int64_t q_row_stride,
                                      const int32_t *table, int64_t table_stride,
                                      const int32_t *lengths, void *out, void *ws,
                                      size_t ws_bytes, void *stream);

/* Which drafted tokens stay, and the token after them, for each of `batch`
 * sequences (speculative sampling: the result is distributed as the target).
 * draft [batch][drafts]: token ids, ended early by a negative one.  target
 * [batch][drafts + 1][vocab]: the target's probabilities before each draft and
 * after the last.  draft_probs [batch][drafts][vocab]: those that the drafts
 * were drawn from, or NULL (each draft certain: probability 1 of itself).
 *   draft i stays while accept_u[b][i] * draft_probs[b][i][x] < target[b][i][x]
 * (in 64 bits).  The token after those that stay is drawn, at the first draft
 * refused, from max(target - draft_probs, 0) (from target where that is 0
 * everywhere), after the last draft from target: the lowest id whose running
 * sum exceeds sample_u[b] times the whole sum.
 * tokens [batch][drafts + 1]: those that stay, the one drawn (-1 if no weight is
 * positive), then -1; accepted [batch]: how many stayed.
 * Probabilities are numbers from 0 to 1 (less, or NaN, counts as 0, more as 1)
 * and are counted in steps of 2^-44, exactly, so that no order of summation
 * decides; their sum need not be 1.  A draft of vocab or more is refused.
 * sample_u: in [0, 1) (less, or NaN, counts as 0, more as the largest below 1). */
typedef struct moeop_verify_config {
    int batch;                   /* 0..65535 */
    int drafts;                  /* 0..31 */
    int vocab;                   /* 1..2^19 */
    int64_t target_stride, draft_stride;  /* elements between rows of vocab */
} moeop_verify_config;

MOE_API moe_status moeop_verify_draft(const moeop_verify_config *cfg, const int32_t *draft,
                                      const float *target, const float *draft_probs,
                                      const float *accept_u, const float *sample_u,
                                      int32_t *tokens, int32_t *accepted, void *stream);

/* Synchronise `stream`, read the current device's status word of these
 * operators into *code (MOE_DEV_*) and clear it.  MOE_DEV_WAIT_TIMEOUT: an
 * on-chip wait exceeded its bound and a product or attention is incomplete.  Returns
 * MOE_ERR_DEVICE_STATUS when the code is non-zero. */
MOE_API moe_status moeop_read_device_status(int *code, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
