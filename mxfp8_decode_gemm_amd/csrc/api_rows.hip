// C ABI of the products of any number of rows: host-side validation (from sizes
// and addresses only, before any HIP call) and dispatch. Declarations, argument
// meanings and error rules are in include/mxrows.h.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/mxrows.h"
#include "rows_internal.h"

using namespace mxg;

namespace {
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
int hip_code(hipError_t e) { return e == hipSuccess ? MXG_OK : MXG_EHIP; }

bool type_ok(int32_t t) { return t == MXG_F32 || t == MXG_BF16 || t == MXG_F16; }
bool format_ok(int32_t f) { return f == MXG_MXFP4 || f == MXG_MXFP8; }
bool x_format_ok(int32_t f) { return format_ok(f) || f == MXG_MXFP8_FAST; }
bool rows_ok(int64_t rows) { return rows >= 1 && rows <= MXG_ROWS_MAX; }
bool weight_ok(int32_t format, int32_t experts, int32_t n, int32_t k) {
  return format_ok(format) && experts >= 1 && experts <= MXG_MOE_MAX_EXPERTS && n >= 8 &&
         n <= MXG_ROWS_MAX_N && n % 8 == 0 && k >= 128 && k <= MXG_ROWS_MAX_K && k % 128 == 0;
}
bool pairs_ok(int32_t tokens, int32_t top_k, int32_t experts) {
  return rows_ok(tokens) && top_k >= 1 && top_k <= MXG_ROUTE_MAX_TOP_K &&
         rows_ok((int64_t)tokens * top_k) && experts >= 1 && experts <= MXG_MOE_MAX_EXPERTS;
}

int64_t packed_expert_bytes(int32_t format, int32_t n, int32_t k) {
  return row_blocks(n) * kb_pairs(k) * 2 * unit_bytes(format);
}
int64_t packed_expert_scale_bytes(int32_t n, int32_t k) { return row_blocks(n) * kb_pairs(k) * 256; }

bool weight_shape_ok(const mxrows_weight* w) {
  return w && weight_ok(w->format, w->experts, w->n, w->k) && (w->gated == 0 || w->gated == 1) &&
         !(w->gated && w->n % 64);
}

// Sizes of a call (the pointers are the caller's to set).
RowsArgs rows_args(const mxrows_weight* w, int32_t x_format, int32_t rows,
                   const int32_t* offsets) {
  RowsArgs a = {};
  a.offsets = offsets;
  a.w_bytes = packed_expert_bytes(w->format, w->n, w->k);
  a.ws_bytes = packed_expert_scale_bytes(w->n, w->k);
  a.experts = w->experts;
  a.n = w->n;
  a.k = w->k;
  a.gated = w->gated;
  a.rows = rows;
  a.fast = x_format == MXG_MXFP8_FAST;
  a.out_n = w->gated ? w->n / 2 : w->n;
  a.nb = (int32_t)row_blocks(w->n);
  a.kp = (int32_t)kb_pairs(w->k);
  return a;
}

RowsChoice choice_of(const mxrows_weight* w, int32_t x_format, int32_t rows, bool grouped) {
  return rows_choice(
      rows_problem(w->format, x_format, w->experts, w->n, w->k, w->gated != 0, rows, grouped));
}

int rows_call(const mxrows_weight* w, int32_t x_format, const uint8_t* x, const uint8_t* x_scale,
              int32_t x_rows, const int32_t* order, int32_t gather, int32_t scatter,
              const int32_t* offsets, int32_t rows, void* workspace, size_t workspace_bytes,
              uint16_t* out, void* stream) {
  if (!w || !w->w || !w->scale || !x || !x_scale || !out) return MXG_EINVAL;
  if (!weight_shape_ok(w) || !x_format_ok(x_format) || !rows_ok(rows)) return MXG_EINVAL;
  if (!aligned(w->w, 16) || !aligned(w->scale, 16) || !aligned(x, 16) || !aligned(x_scale, 4) ||
      !aligned(out, 16))
    return MXG_EALIGN;
  if (w->format == MXG_MXFP8 && x_format == MXG_MXFP4) return MXG_EUNSUPPORTED;
  const int64_t x_row = x_format == MXG_MXFP4 ? w->k / 2 : w->k;
  if (gather && (int64_t)x_rows * x_row >= ((int64_t)1 << 32)) return MXG_EUNSUPPORTED;
  RowsArgs a = rows_args(w, x_format, rows, offsets);
  a.w = w->w;
  a.ws = w->scale;
  a.x = x;
  a.xs = x_scale;
  a.out = out;
  a.order = order;
  a.x_rows = x_rows;
  a.gather = gather;
  a.over = gather_quotient(gather);
  a.scatter = scatter;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const RowsChoice c = choice_of(w, x_format, rows, offsets != nullptr);
  if (c.side == 0) return hip_code(launch_rows_stream(a, w->format, x_format, s));
  const size_t needed = choice_workspace(c);
  if (needed) {
    if (!workspace || workspace_bytes < needed) return MXG_EWORKSPACE;
    if (!aligned(workspace, 16)) return MXG_EALIGN;
    a.partial = static_cast<float*>(workspace);
  }
  return hip_code(launch_rows_tile(a, w->format, x_format, c, s));
}
}  // namespace

extern "C" {

int mxfp4_quantize(const void* x, int32_t x_type, int64_t row_stride, int32_t rows, int32_t k,
                   uint8_t* x_q, uint8_t* x_scale, void* stream) {
  if (!x || !x_q || !x_scale || !type_ok(x_type) || !rows_ok(rows)) return MXG_EINVAL;
  if (k < 32 || k > MXG_ROWS_MAX_K || k % 32) return MXG_EINVAL;
  if (row_stride < k || row_stride > ((int64_t)1 << 31) ||
      row_stride % (x_type == MXG_F32 ? 4 : 8))
    return MXG_EINVAL;
  if (!aligned(x, 16) || !aligned(x_q, 16)) return MXG_EALIGN;
  return hip_code(launch_fp4_quantize(x, x_type, row_stride, rows, k, x_q, x_scale,
                                      static_cast<hipStream_t>(stream)));
}

int mxfp4_dequantize(const uint8_t* x_q, const uint8_t* x_scale, int32_t rows, int32_t k,
                     int32_t y_type, void* y, void* stream) {
  if (!x_q || !x_scale || !y || !type_ok(y_type) || !rows_ok(rows)) return MXG_EINVAL;
  if (k < 32 || k > MXG_ROWS_MAX_K || k % 32) return MXG_EINVAL;
  if (!aligned(x_q, 16) || !aligned(y, 16)) return MXG_EALIGN;
  return hip_code(launch_fp4_dequantize(x_q, x_scale, rows, k, y_type, y,
                                        static_cast<hipStream_t>(stream)));
}

size_t mxrows_packed_weight_bytes(int32_t format, int32_t experts, int32_t n, int32_t k) {
  if (!weight_ok(format, experts, n, k)) return 0;
  return (size_t)experts * packed_expert_bytes(format, n, k);
}

size_t mxrows_packed_scale_bytes(int32_t format, int32_t experts, int32_t n, int32_t k) {
  if (!weight_ok(format, experts, n, k)) return 0;
  return (size_t)experts * packed_expert_scale_bytes(n, k);
}

int mxrows_pack_weight(int32_t format, const uint8_t* w, const uint8_t* w_scale, int32_t experts,
                       int32_t n, int32_t k, uint8_t* w_packed, uint8_t* ws_packed, void* stream) {
  if (!w || !w_scale || !w_packed || !ws_packed) return MXG_EINVAL;
  if (!weight_ok(format, experts, n, k)) return MXG_EINVAL;
  if (!aligned(w, 16) || !aligned(w_scale, 4) || !aligned(w_packed, 16) || !aligned(ws_packed, 16))
    return MXG_EALIGN;
  return hip_code(launch_rows_pack(format, w, w_scale, experts, n, k, w_packed, ws_packed,
                                   static_cast<hipStream_t>(stream)));
}

size_t mxrows_workspace_bytes(const mxrows_weight* w, int32_t x_format, int32_t rows) {
  if (!weight_shape_ok(w) || w->experts != 1 || !x_format_ok(x_format) || !rows_ok(rows))
    return 0;
  return choice_workspace(choice_of(w, x_format, rows, false));
}

int mxrows_product(const mxrows_weight* w, int32_t x_format, const uint8_t* x,
                   const uint8_t* x_scale, int32_t rows, void* workspace, size_t workspace_bytes,
                   uint16_t* out, void* stream) {
  if (w && w->experts != 1) return MXG_EINVAL;
  return rows_call(w, x_format, x, x_scale, rows, nullptr, 0, 0, nullptr, rows, workspace,
                   workspace_bytes, out, stream);
}

size_t mxmoe_sort_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts) {
  if (!pairs_ok(tokens, top_k, experts)) return 0;
  return sort_workspace((int64_t)tokens * top_k, experts);
}

int mxmoe_sort(const int32_t* ids, int32_t tokens, int32_t top_k, int32_t experts,
               void* workspace, size_t workspace_bytes, int32_t* order, int32_t* offsets,
               void* stream) {
  if (!ids || !order || !offsets || !pairs_ok(tokens, top_k, experts)) return MXG_EINVAL;
  if (!aligned(ids, 4) || !aligned(order, 4) || !aligned(offsets, 4)) return MXG_EALIGN;
  const size_t needed = mxmoe_sort_workspace_bytes(tokens, top_k, experts);
  if (needed && (!workspace || workspace_bytes < needed)) return MXG_EWORKSPACE;
  if (!aligned(workspace, 16)) return MXG_EALIGN;
  return hip_code(launch_sort(ids, tokens * top_k, experts, workspace, order, offsets,
                              static_cast<hipStream_t>(stream)));
}

int mxmoe_grouped(const mxrows_weight* w, int32_t x_format, const uint8_t* x,
                  const uint8_t* x_scale, int32_t x_rows, const int32_t* order, int32_t gather,
                  int32_t scatter, const int32_t* offsets, int32_t rows, uint16_t* out,
                  void* stream) {
  if (!offsets || gather < 0 || gather > MXG_ROUTE_MAX_TOP_K || (scatter != 0 && scatter != 1)) return MXG_EINVAL;
  if ((gather || scatter) && !order) return MXG_EINVAL;
  if (!rows_ok(x_rows) || (!gather && x_rows != rows)) return MXG_EINVAL;
  if (!aligned(offsets, 4) || !aligned(order, 4)) return MXG_EALIGN;
  return rows_call(w, x_format, x, x_scale, x_rows, order, gather, scatter, offsets, rows, nullptr,
                   0, out, stream);
}

int mxmoe_combine(const uint16_t* y, const int32_t* ids, const float* weights, int32_t tokens,
                  int32_t top_k, int32_t experts, int32_t hidden, uint16_t* out, void* stream) {
  if (!y || !ids || !weights || !out || !pairs_ok(tokens, top_k, experts)) return MXG_EINVAL;
  if (hidden < 8 || hidden > MXG_ROWS_MAX_N || hidden % 8) return MXG_EINVAL;
  if (!aligned(y, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(out, 16))
    return MXG_EALIGN;
  return hip_code(launch_combine(y, ids, weights, tokens, top_k, experts, hidden, out,
                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
