/*
 * mxdecode.h -- C ABI of the decode operators whose weights are chosen per
 * row, on the same library, packed weights and mailbox as mxgemm.h:
 *
 *   mxmoe_route     expert routing: scores, balance bias, groups, top-k
 *   mxmoe_experts   the gated MXFP8 products of the chosen experts
 *   mxgemm_lora     the MXFP8 projection with each row's low-rank adapter
 *
 * Conventions are those of mxgemm.h: device pointers owned by the caller, all
 * work enqueued on `stream` without a host synchronization, arguments checked
 * on the host from sizes and addresses alone before anything is enqueued, a
 * negative MXG_E* code on error (mxg_strerror describes it). Every call may be
 * captured into a HIP graph. The pointers belong to the device that is current
 * at the call, and `stream` to the same device. Outputs never overlap inputs.
 */
#ifndef MXDECODE_H
#define MXDECODE_H

#include <stddef.h>
#include <stdint.h>

#include "mxgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- expert routing ----------------------------------------------------- */

#define MXG_ROUTE_SOFTMAX 0
#define MXG_ROUTE_SIGMOID 1
#define MXG_F32 0             /* type of the logits */
#define MXG_BF16 1
#define MXG_ROUTE_MAX_EXPERTS 1024
#define MXG_ROUTE_MAX_GROUPS 64
#define MXG_ROUTE_MAX_TOP_K 32

/* What a router does with a row of logits (plain data on the host). */
typedef struct mxmoe_router {
  int32_t experts;     /* 1..MXG_ROUTE_MAX_EXPERTS */
  int32_t top_k;       /* 1..MXG_ROUTE_MAX_TOP_K, at most the experts of
                          top_groups groups */
  int32_t score;       /* MXG_ROUTE_SOFTMAX (over all experts) or _SIGMOID */
  int32_t groups;      /* 1..MXG_ROUTE_MAX_GROUPS, divides experts: group g
                          holds the experts g * experts / groups and on */
  int32_t top_groups;  /* 1..groups: the groups a row may choose from */
  int32_t group_best;  /* 1 or 2: a group's score is the sum of that many of
                          its largest choices */
  int32_t renormalize; /* 0, or 1: a row's weights are divided by their sum */
  float scale;         /* every weight is multiplied by it */
} mxmoe_router;

/* Routes `tokens` rows of logits. Per row, with score s[e] the softmax over
 * all experts or the sigmoid of logit e, and choice c[e] = s[e] + bias[e]
 * (s[e] without a bias):
 *   - the top_groups groups of the largest group score are kept;
 *   - ids[t][j], j = 0..top_k-1, are the experts of the largest choices in
 *     the kept groups, in descending order;
 *   - weights[t][j] = s[ids[t][j]], divided by their sum when renormalize is
 *     set, times scale: the bias counts for the choice only.
 * Choices and group scores are compared as 64-bit values (a score below
 * 2^-1022 is zero); equal ones go to the lowest index, also those of different
 * logits (sigmoids of neighbours from about 23 on, logits less than 2^-53
 * apart). Weights are rounded to 32 bits from scores that keep their bits: small
 * ones (below exp(-64) of the largest) are 64-bit values.
 *
 * An expert whose logit is -infinity or NaN is out: it is never chosen and
 * adds nothing to the softmax or to its group. A bias of -infinity or NaN
 * keeps its expert from being chosen. Where fewer than top_k
 * experts are left, the rest of the row is id -1 with weight 0, which
 * mxmoe_experts passes over. A sum of weights of zero leaves them zero. With
 * softmax, logits of +infinity share the row's weight.
 *
 *   logits      device, [tokens] rows of `experts` values, row t at
 *               logits + t * row_stride elements; type MXG_F32 or MXG_BF16,
 *               aligned to its element
 *   row_stride  elements, from experts to 2^31
 *   bias        device or NULL: [experts] FP32
 *   tokens      rows, 1..2^24
 *   ids         device, [tokens][top_k] int32
 *   weights     device, [tokens][top_k] FP32
 * Errors: MXG_EINVAL, MXG_EALIGN (a pointer not aligned to its element),
 * MXG_EHIP. */
int mxmoe_route(const mxmoe_router* router, const void* logits, int32_t logits_type,
                int64_t row_stride, const float* bias, int32_t tokens, int32_t* ids,
                float* weights, void* stream);

/* ---- the chosen experts' products ---------------------------------------- */

#define MXG_MOE_MAX_EXPERTS 1024
#define MXG_MOE_MAX_PAIRS 1024 /* tokens * top_k of one call */

/* Bytes of `experts` weights [n, k] in the packed layout: expert e's weight is
 * mxgemm_pack_weight's, at e * mxgemm_packed_weight_bytes(n, k), its scales at
 * e * mxgemm_packed_scale_bytes(n, k). 0 on bad sizes. */
size_t mxmoe_packed_weight_bytes(int32_t experts, int32_t n, int32_t k);
size_t mxmoe_packed_scale_bytes(int32_t experts, int32_t n, int32_t k);

/* Packs row-major w [experts, n, k] (e4m3fn) and w_scale [experts, n, k/32]
 * (E8M0). experts 1..MXG_MOE_MAX_EXPERTS, n % 16 == 0, k % 128 == 0; all four
 * pointers device, 16-B aligned. Errors: MXG_EINVAL, MXG_EALIGN, MXG_EHIP. */
int mxmoe_pack_weight(const uint8_t* w, const uint8_t* w_scale, int32_t experts, int32_t n,
                      int32_t k, uint8_t* w_packed, uint8_t* ws_packed, void* stream);

/* Bytes of workspace mxmoe_experts needs for these sizes; 0 on bad sizes. It
 * needs no arming, and holds nothing from one call to the next. A workspace
 * serves every call of these experts, hidden and inter with as many pairs (tokens *
 * top_k) or fewer. */
size_t mxmoe_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts, int32_t hidden,
                             int32_t inter);

/* The gated product of the chosen experts:
 *
 *   h[t, j]  = silu(Wg[e] x[t]) * (Wu[e] x[t])        e = ids[t][j]
 *   out[t]   = sum_j weights[t][j] * W2[e] h[t, j]
 *
 * with W13[e] = [Wg[e]; Wu[e]] of [2 inter, hidden] and W2[e] of [hidden,
 * inter], and silu(v) = v / (1 + exp(-v)). An id outside 0..experts-1 adds
 * nothing; a row without any expert comes out as zeros. A row may name an
 * expert more than once. Products accumulate in FP32, h is held as the sum of
 * two BF16 values (to 2^-18 of itself or 2^-134; beyond BF16's range it is
 * infinite), the sum over j runs in FP32 in ascending order, and the result is
 * rounded once to BF16. A weight is the BF16 value nearest to its code times its
 * scale: exact for scale bytes 3..246 (255 is the E8M0 NaN and not taken); one
 * beyond BF16's range is infinite, and in w2 makes NaN of its column. Results are
 * the same bits on every call.
 *
 *   x         device, [tokens, hidden] BF16, 16-B aligned
 *   ids       device, [tokens, top_k] int32
 *   weights   device, [tokens, top_k] FP32
 *   w13, w13_scale, w2, w2_scale  device, packed by mxmoe_pack_weight, 16-B
 *             aligned
 *   tokens, top_k  >= 1, tokens * top_k <= MXG_MOE_MAX_PAIRS
 *   experts   1..MXG_MOE_MAX_EXPERTS
 *   hidden, inter  positive multiples of 128, at most 32768
 *   workspace device, at least mxmoe_workspace_bytes(), 16-B aligned; one call
 *             at a time per workspace
 *   out       device, [tokens, hidden] BF16, 16-B aligned
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EWORKSPACE, MXG_EHIP. */
int mxmoe_experts(const uint16_t* x, const int32_t* ids, const float* weights,
                  const uint8_t* w13, const uint8_t* w13_scale, const uint8_t* w2,
                  const uint8_t* w2_scale, int32_t tokens, int32_t top_k, int32_t experts,
                  int32_t hidden, int32_t inter, void* workspace, size_t workspace_bytes,
                  uint16_t* out, void* stream);

/* ---- the projection with per-row adapters -------------------------------- */

#define MXG_LORA_MAX_RANK 128

/* The adapters of one projection W [n, k] (plain data on the host). Adapters of
 * a smaller rank than the stack's are padded with zero rows of a. */
typedef struct mxg_lora {
  const uint16_t* a;    /* device, [adapters, rank, k] BF16, 16-B aligned */
  const uint16_t* b;    /* device, [adapters, n, rank] BF16, 16-B aligned */
  const float* scale;   /* device, [adapters] FP32 */
  const int32_t* ids;   /* device, [m]: each row's adapter; outside
                           0..adapters-1: none */
  int32_t adapters;     /* >= 1 */
  int32_t rank;         /* a multiple of 8, 8..MXG_LORA_MAX_RANK */
} mxg_lora;

/* Bytes of scratch mxgemm_lora needs for n columns, beside the split-K
 * workspace; 0 on bad sizes. The workgroups exchange A[i] x through it as
 * (value, epoch) pairs, like the split-K partials in theirs. */
size_t mxgemm_lora_scratch_bytes(int32_t n);

/* Arm a scratch: once before first use, outside capture; it then serves calls
 * of any size up to its own, in any order. scratch_bytes: at least
 * mxgemm_lora_scratch_bytes(8), a multiple of 16. Errors: MXG_EINVAL,
 * MXG_EALIGN, MXG_EHIP. */
int mxgemm_lora_scratch_init(void* scratch, size_t scratch_bytes, void* stream);

/* The projection of mxgemm_publish, mxgemm_publish_bf16 or mxgemm with a
 * low-rank adapter beside it, chosen per row:
 *
 *   C[t] = W q(x)[t] + scale[i] * B[i] (A[i] x[t])          i = ids[t]
 *
 * The shared product is theirs (with BF16 x: of the quantized activation);
 * the adapter takes BF16 x as it is, MXFP8 x as the values it stands for.
 * Both products of the adapter accumulate in FP32, u = scale[i] A[i] x between
 * them is held as the sum of two BF16 values (to 2^-18 of itself or 2^-134; an
 * infinity in B therefore makes NaN of its column), and the result is added to the
 * shared product before the one rounding to BF16.
 *
 *   mb       a mailbox to publish C into (then collect it, as after
 *            mxgemm_publish), or NULL for the plain product into c_out
 *   x, x_scale  MXFP8 x, or both NULL with x_bf16 given
 *   x_bf16   BF16 x, or NULL with x and x_scale given
 *   scratch  device, at least mxgemm_lora_scratch_bytes(n), 16-B aligned, armed
 *            by mxgemm_lora_scratch_init; one call at a time per scratch
 *   c_out    device [m, n] BF16 as rounded; may be NULL with mb
 * Other arguments as mxgemm_publish. With split_k > 1 the workgroups of a call
 * wait for each other, as there: two such calls must not run at once on one
 * device.
 *
 * Failure: workgroup 0 gives up waiting for the others to start after
 * mb->spin_limit polls (MXG_DEFAULT_SPIN_LIMIT without mb) and sets
 * MXG_ERR_SPLITK_SPIN in the scratch's ERROR word (MXG_WS_ERROR): the call and
 * later ones are right, but slow until the scratch is armed again. A split-K
 * wait that gives up sets it in the split-K workspace's ERROR word, as in
 * mxgemm_publish: the values it was for, and all of later calls' on that
 * workspace until it is armed again, are NaN in c_out and unpublished.
 * Errors: its errors (MXG_EUNSUPPORTED also where the x slice leaves no
 * LDS for u), MXG_EINVAL for a bad adapter argument, MXG_EWORKSPACE for a missing
 * or small scratch. */
int mxgemm_lora(const mxg_mailbox* mb, const uint8_t* w, const uint8_t* w_scale,
                const uint8_t* x, const uint8_t* x_scale, const uint16_t* x_bf16, int32_t m,
                int32_t n, int32_t k, int32_t split_k, void* workspace, size_t workspace_bytes,
                const mxg_lora* lora, void* scratch, size_t scratch_bytes, uint16_t* c_out,
                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXDECODE_H */
