/*
 * mxrows.h -- C ABI of the products of any number of rows, on the same library
 * as mxgemm.h and mxdecode.h: MXFP4 beside MXFP8, a prompt's rows beside a
 * decode step's.
 *
 *   mxfp4_quantize, mxfp4_dequantize   rows to MXFP4 and back
 *   mxrows_product                     C[t] = W x[t], W and x in MXFP4 or MXFP8
 *   mxmoe_sort                         a router's pairs by expert
 *   mxmoe_grouped                      the same product, each expert's on its rows
 *   mxmoe_combine                      the weighted sum of a token's pairs
 *
 * MXFP4: E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 with a sign in bit 3), two in a
 * byte, the lower index in the low half, with one E8M0 scale byte per 32 values
 * along K. MXFP8: e4m3fn codes with the same scales. Row-major: k/2 or k bytes
 * and k/32 scale bytes a row.
 *
 * Conventions are those of mxgemm.h: device pointers owned by the caller, all
 * work enqueued on `stream` without a host synchronization, arguments checked
 * on the host from sizes and addresses alone before anything is enqueued, a
 * negative MXG_E* code on error (mxg_strerror describes it). Every call may be
 * captured into a HIP graph. The pointers belong to the device that is current
 * at the call, and `stream` to the same device. Outputs never overlap inputs.
 * Nothing is kept from one call to the next, and results are the same bits on
 * every call.
 */
#ifndef MXROWS_H
#define MXROWS_H

#include <stddef.h>
#include <stdint.h>

#include "mxdecode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of values beside MXG_F32 and MXG_BF16, and formats of codes. */
#define MXG_F16 2
#define MXG_MXFP4 4
#define MXG_MXFP8 8
#define MXG_MXFP8_FAST 9 /* as x_format: MXFP8 rows, sums of fewer bits (mxrows_product) */

#define MXG_ROWS_MAX 16777216  /* rows of a call (2^24) */
#define MXG_ROWS_MAX_N 1048576 /* rows of a weight */
#define MXG_ROWS_MAX_K 65536

/* ---- MXFP4 ---------------------------------------------------------------- */

/* Rows to MXFP4: per 32 consecutive values along K, e = the smallest integer
 * with max|x| <= 6 * 2^e, clamped to [-127, 127] (an all-zero block: -127), scale
 * byte e + 127, and each code the E2M1 value nearest to x / 2^e (ties to even,
 * sign kept). A block holding an infinity or NaN gets scale byte 0xFF (the E8M0
 * NaN) and codes 7 | sign. The rule is mxfp8_quantize's.
 *   x          device, `rows` rows of k values, row t at x + t * row_stride
 *              elements; type MXG_F32, MXG_BF16 or MXG_F16, 16-B aligned
 *   row_stride elements, from k to 2^31, a multiple of 16 bytes
 *   rows, k    1..MXG_ROWS_MAX; a multiple of 32, at most MXG_ROWS_MAX_K
 *   x_q        device, [rows, k/2], 16-B aligned
 *   x_scale    device, [rows, k/32]
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EHIP. */
int mxfp4_quantize(const void* x, int32_t x_type, int64_t row_stride, int32_t rows, int32_t k,
                   uint8_t* x_q, uint8_t* x_scale, void* stream);

/* The values that codes and scales stand for, rounded to the type (exact in FP32
 * and BF16 for scale bytes 0..252; beyond a type's range they are infinite, and
 * the scale byte 255 makes NaN).
 *   x_q, x_scale  as mxfp4_quantize writes them
 *   y          device, [rows, k] of type MXG_F32, MXG_BF16 or MXG_F16, 16-B aligned
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EHIP. */
int mxfp4_dequantize(const uint8_t* x_q, const uint8_t* x_scale, int32_t rows, int32_t k,
                     int32_t y_type, void* y, void* stream);

/* ---- weights -------------------------------------------------------------- */

/* Bytes of a stack of `experts` weights [n, k] (1 for a plain one) in the packed
 * layout of these products: MXG_MXFP4 or MXG_MXFP8 codes in the order in which
 * the matrix instructions take them, n padded to 32 and k to 256 with zeros. 0
 * on bad sizes: experts 1..MXG_MOE_MAX_EXPERTS, n a multiple of 8 up to
 * MXG_ROWS_MAX_N, k a multiple of 128 up to MXG_ROWS_MAX_K. */
size_t mxrows_packed_weight_bytes(int32_t format, int32_t experts, int32_t n, int32_t k);
size_t mxrows_packed_scale_bytes(int32_t format, int32_t experts, int32_t n, int32_t k);

/* Packs row-major codes w [experts, n, k] and w_scale [experts, n, k/32]; all
 * four pointers device, 16-B aligned (w_scale: 4-B). Errors: MXG_EINVAL,
 * MXG_EALIGN, MXG_EHIP. */
int mxrows_pack_weight(int32_t format, const uint8_t* w, const uint8_t* w_scale, int32_t experts,
                       int32_t n, int32_t k, uint8_t* w_packed, uint8_t* ws_packed, void* stream);

/* A packed stack of weights (plain data on the host). */
typedef struct mxrows_weight {
  const uint8_t* w;       /* device, of mxrows_pack_weight, 16-B aligned */
  const uint8_t* scale;   /* device, the same */
  int32_t format;         /* MXG_MXFP4 or MXG_MXFP8 */
  int32_t experts, n, k;  /* as packed */
  int32_t gated;          /* 0, or 1: the rows are [gate; up] of n/2 each, and the
                             product is silu(Wg x) * (Wu x), n/2 wide, with
                             silu(v) = v / (1 + exp(-v)); n a multiple of 64 */
} mxrows_weight;

/* ---- the product ----------------------------------------------------------- */

/* Bytes of workspace mxrows_product needs for `rows` rows of this weight (its
 * pointers are not looked at): 0 where K is not divided among workgroups, at most
 * 16 MiB, and 0 on bad sizes. It needs no arming. */
size_t mxrows_workspace_bytes(const mxrows_weight* w, int32_t x_format, int32_t rows);

/* out[t] = W x[t] for t in 0..rows-1, rounded once to BF16; gated:
 * silu(Wg x[t]) * (Wu x[t]), formed in FP32 before the rounding. A row is out_n =
 * n (gated: n/2) values.
 *
 * Sums are FP32 and keep what FP32 keeps. MXFP4 by MXFP4 goes through the matrix
 * instructions as codes and scales lie, eight aligned products of K at a time, whose sum
 * is exact. With MXFP8 rows the operands are taken to BF16 with their scales, which is
 * exact for scale bytes 3..246 (mxgemm's contraction). Where a nonzero code has another
 * scale byte, the 64 values of K around it go by the scaled instruction instead, for at
 * most 64 rows of W and of x together; that loses, of each eight aligned products, what
 * lies below 2^-13 of the largest (toward zero). Rows of MXG_MXFP8_FAST all go by it, up
 * to twice as fast for many rows: each eight products may be off by 7 * 2^-13 of the
 * largest of them, so that a result is as good as its BF16 rounding unless its sum
 * cancels to less than its products. Products and sums below 2^-149 are lost, a result or partial sum beyond the
 * FP32 range is infinite or NaN, and a scale byte 255 or an e4m3fn NaN makes NaN of what
 * it enters.
 *
 *   w         with experts == 1
 *   x_format  MXG_MXFP4 (with an MXFP4 weight), MXG_MXFP8 or MXG_MXFP8_FAST
 *   x, x_scale  device, [rows, k] codes (16-B aligned), [rows, k/32] (4-B)
 *   rows      1..MXG_ROWS_MAX
 *   workspace device, at least mxrows_workspace_bytes(), 16-B aligned; one call at
 *             a time per workspace. NULL where that is 0
 *   out       device, [rows, out_n] BF16, 16-B aligned
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EWORKSPACE, MXG_EUNSUPPORTED (an MXFP8
 * weight on MXFP4 x), MXG_EHIP. */
int mxrows_product(const mxrows_weight* w, int32_t x_format, const uint8_t* x,
                   const uint8_t* x_scale, int32_t rows, void* workspace, size_t workspace_bytes,
                   uint16_t* out, void* stream);

/* ---- a router's pairs by expert -------------------------------------------- */

/* Bytes of workspace mxmoe_sort needs: 0 for at most 4096 pairs, and on bad
 * sizes. It needs no arming. */
size_t mxmoe_sort_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts);

/* The pairs p = t * top_k + j of a router's choices by expert, an expert's in
 * ascending order: order[offsets[e] .. offsets[e + 1]) are the pairs with
 * ids[p] == e. Pairs without an expert (an id outside 0..experts-1) come after
 * offsets[experts], in ascending order, so that order is a permutation.
 *   ids       device, [tokens, top_k] int32, as mxmoe_route writes them
 *   tokens    1..MXG_ROWS_MAX; top_k 1..MXG_ROUTE_MAX_TOP_K; at most
 *             MXG_ROWS_MAX pairs
 *   experts   1..MXG_MOE_MAX_EXPERTS
 *   workspace device, at least mxmoe_sort_workspace_bytes(), 16-B aligned; one
 *             call at a time per workspace. NULL where that is 0
 *   order     device, [tokens * top_k] int32
 *   offsets   device, [experts + 1] int32
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EWORKSPACE, MXG_EHIP. */
int mxmoe_sort(const int32_t* ids, int32_t tokens, int32_t top_k, int32_t experts,
               void* workspace, size_t workspace_bytes, int32_t* order, int32_t* offsets,
               void* stream);

/* ---- the product grouped by expert ----------------------------------------- */

/* out[o(i)] = W[e] x[r(i)] for the sorted rows i in offsets[e] ..
 * offsets[e + 1] - 1 of every expert e, with the arithmetic of mxrows_product;
 *   r(i) = order[i] / gather with gather from 1 to MXG_ROUTE_MAX_TOP_K (a router's
 *          tokens: its top_k), i with gather 0;
 *   o(i) = order[i] with scatter 1, i with scatter 0.
 * An expert may have no rows. Rows of out that no i leads to (the pairs without
 * an expert) are left as they were.
 *
 *   w         experts weights
 *   x_rows    rows of x: r(i) lies in 0..x_rows-1. With gather 0, equal to rows.
 *             With gather, x and x_scale take less than 4 GiB
 *             (MXG_EUNSUPPORTED otherwise).
 *   order     device, [rows] int32, or NULL with gather and scatter 0; its values
 *             name rows of x and out, those of out each at most once. One that
 *             leads outside x gives the row a value that says nothing, one outside
 *             out is not written.
 *   offsets   device, [experts + 1] int32, ascending, within 0..rows; parts
 *             outside are passed over
 *   rows      1..MXG_ROWS_MAX: rows of order and of out
 * Other arguments and errors as mxrows_product (no workspace). */
int mxmoe_grouped(const mxrows_weight* w, int32_t x_format, const uint8_t* x,
                  const uint8_t* x_scale, int32_t x_rows, const int32_t* order, int32_t gather,
                  int32_t scatter, const int32_t* offsets, int32_t rows, uint16_t* out,
                  void* stream);

/* ---- the sum over a token's pairs -------------------------------------------- */

/* out[t] = sum_j weights[t, j] * y[t, j] over the pairs whose id is an expert, in
 * FP32, in ascending order, rounded once to BF16; rows of y without an expert are
 * not read, a token without any comes out as zeros.
 *   y         device, [tokens, top_k, hidden] BF16, 16-B aligned
 *   ids, weights  device, [tokens, top_k] int32, FP32
 *   tokens    1..MXG_ROWS_MAX; top_k 1..MXG_ROUTE_MAX_TOP_K; at most
 *             MXG_ROWS_MAX pairs
 *   hidden    a multiple of 8, 8..MXG_ROWS_MAX_N
 *   out       device, [tokens, hidden] BF16, 16-B aligned
 * Errors: MXG_EINVAL, MXG_EALIGN, MXG_EHIP. */
int mxmoe_combine(const uint16_t* y, const int32_t* ids, const float* weights, int32_t tokens,
                  int32_t top_k, int32_t experts, int32_t hidden, uint16_t* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXROWS_H */
