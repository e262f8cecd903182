// Internal declarations of the products of any number of rows
// (include/mxrows.h). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mxrows.h"
#include "gather_quotient.h"
#include "rows_choice.h"

namespace mxg {

// The packed weight (mxrows_pack_weight). Unit (rb, kb): 32 rows by 128 values
// of K, two MFMA steps s of 64. Lane l of a wave holds row l % 32; with g = l /
// 32, step s takes from it
//   MXFP4: the 16 bytes of K block 2 s + g               at s 1024 + 16 l
//   MXFP8: the 16-byte pieces 4 s + g and 4 s + 2 + g    at s 2048 + 16 l, + 1024
// (of the unit's four 32-wide blocks, eight pieces), and as its scale that of
// block 2 s + g either way: the instruction's own order of K. Units lie [row
// block][kb], 2048 or 4096 bytes each; scales [row block][kb / 2][lane] as words,
// byte 2 (kb % 2) + s. kb runs to an even number, rows to 32: zeros with scale
// byte 127. (Sizes: rows_choice.h.)
struct RowsArgs {
  const uint8_t *w, *ws;  // packed
  const uint8_t *x, *xs;  // row-major codes and scales
  uint16_t* out;          // [*, out_n] BF16
  const int32_t* offsets; // [experts + 1], or null: one weight, all rows
  const int32_t* order;   // or null
  int64_t w_bytes, ws_bytes;  // of one expert
  int32_t experts, n, k, gated, rows, x_rows, gather, scatter;
  int32_t fast;           // MXG_MXFP8_FAST
  int32_t out_n, nb, kp;  // columns of out; row blocks of a weight, pairs of kb
  GatherQuotient over;    // of gather, from 2 on
  float* partial;         // workspace of a split K (one weight, all rows), or null
};

hipError_t launch_rows_stream(const RowsArgs& a, int w_format, int x_format, hipStream_t s);
// By tiles; choice_workspace(h) bytes of a.partial are used.
hipError_t launch_rows_tile(const RowsArgs& a, int w_format, int x_format, const RowsChoice& h,
                            hipStream_t s);
// Its tiles for MXFP8 rows that are not to be `fast` (rows_bf16.hip).
hipError_t launch_rows_bf16(const RowsArgs& a, int w_format, int row_tiles, int col_tiles,
                            int split, hipStream_t s);

hipError_t launch_rows_pack(int format, const uint8_t* w, const uint8_t* ws, int experts, int n,
                            int k, uint8_t* wp, uint8_t* wsp, hipStream_t s);

hipError_t launch_fp4_quantize(const void* x, int x_type, int64_t row_stride, int rows, int k,
                               uint8_t* xq, uint8_t* xs, hipStream_t s);
hipError_t launch_fp4_dequantize(const uint8_t* xq, const uint8_t* xs, int rows, int k, int y_type,
                                 void* y, hipStream_t s);

size_t sort_workspace(int64_t pairs, int experts);
hipError_t launch_sort(const int32_t* ids, int pairs, int experts, void* workspace, int32_t* order,
                       int32_t* offsets, hipStream_t s);

hipError_t launch_combine(const uint16_t* y, const int32_t* ids, const float* weights, int tokens,
                          int top_k, int experts, int hidden, uint16_t* out, hipStream_t s);

}  // namespace mxg
