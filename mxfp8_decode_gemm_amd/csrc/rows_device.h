// Device helpers shared by the kernels of the products of any number of rows
// (gfx950): the scaled MFMA by format, where a tile of rows lies, the epilogue's
// arithmetic.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rows_internal.h"

namespace mxg {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// The operand of one MFMA step: 32 rows by 64 values of K, 16 or 32 bytes a lane.
template <int FORMAT>
struct Piece {
  v4u lo, hi;
};
template <>
struct Piece<MXG_MXFP4> {
  v4u lo;
};

template <int FORMAT>
__device__ __forceinline__ v8i operand(const Piece<FORMAT>& p) {
  if constexpr (FORMAT == MXG_MXFP4)
    return v8i{(int)p.lo.x, (int)p.lo.y, (int)p.lo.z, (int)p.lo.w, 0, 0, 0, 0};
  else
    return v8i{(int)p.lo.x, (int)p.lo.y, (int)p.lo.z, (int)p.lo.w,
               (int)p.hi.x, (int)p.hi.y, (int)p.hi.z, (int)p.hi.w};
}

// acc[n][t] += sum over 64 K of W[n] x[t], byte BW of sw and byte BX of sx the
// lane's scales. acc: lane l holds column t = l % 32 and the rows n = 8 (i / 4) +
// 4 (l / 32) + i % 4.
template <int FW, int FX, int BW, int BX>
__device__ __forceinline__ v16f product(const Piece<FW>& w, uint32_t sw, const Piece<FX>& x,
                                        uint32_t sx, v16f acc) {
  constexpr int CW = FW == MXG_MXFP4 ? 4 : 0, CX = FX == MXG_MXFP4 ? 4 : 0;  // E2M1, e4m3
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand<FW>(w), operand<FX>(x), acc, CW,
                                                         CX, BW, (int)sw, BX, (int)sx);
}

// silu(gate) * up. With E = exp(-|gate|), silu is gate / (1 + E) for a gate from zero
// on and gate E / (1 + E) below: the reciprocal's argument lies in 1..2, and E as the
// square of exp2(-|gate| log2(e) / 2) is right down to FP32's subnormals. E is off by
// |gate| 2^-23 and a few 2^-24 of itself (the exponent's rounding), far below the
// result's BF16 rounding; expf and a division took twice the time of a tile's
// epilogue.
__device__ __forceinline__ float gated(float gate, float up) {
  const float q = __builtin_amdgcn_exp2f(fabsf(gate) * -0.72134752f);
  const float e = q * q;
  return gate * (gate < 0.f ? e : 1.f) * __builtin_amdgcn_rcpf(1.f + e) * up;
}

// Eight neighbouring columns of lane l's row l % 32 in BF16, from the values that it
// holds of 16: v[0..3] are columns 4 (l / 32) .. and v[4..7] those 8 on; a lane's four
// meet those of the lane 32 on, and lane group l / 32 gets columns 8 (l / 32) ...
template <typename V>
__device__ __forceinline__ uint4 eight_columns(const V& v, int q = 0) {
  const auto lo = __builtin_amdgcn_permlane32_swap(bf16_pair(v[4 * q], v[4 * q + 1]),
                                                   bf16_pair(v[4 * q + 4], v[4 * q + 5]), false,
                                                   false);
  const auto hi = __builtin_amdgcn_permlane32_swap(bf16_pair(v[4 * q + 2], v[4 * q + 3]),
                                                   bf16_pair(v[4 * q + 6], v[4 * q + 7]), false,
                                                   false);
  return uint4{lo[0], hi[0], lo[1], hi[1]};
}

__device__ __forceinline__ v16f gated(const v16f& gate, const v16f& up) {
  v16f h;
#pragma unroll
  for (int q = 0; q < 16; ++q) h[q] = gated(gate[q], up[q]);
  return h;
}

// A tile of sorted rows of one expert: rows r0 .. r1 - 1; expert -1: no such tile.
struct RowTile {
  int expert, r0, r1;
};

// Tile number `at` of TILE rows, counted over the experts in turn. Every lane of
// the wave takes part; the result is wave-uniform.
template <int TILE>
__device__ __forceinline__ RowTile find_tile(const int32_t* offsets, int experts, int rows, int at,
                                             int lane) {
  const int per = (experts + 63) >> 6;  // consecutive experts of a lane
  int own = 0;
  for (int j = 0; j < per; ++j) {
    const int e = lane * per + j;
    if (e < experts) {
      const int a = max(offsets[e], 0), b = min(offsets[e + 1], rows);
      own += b > a ? (b - a + TILE - 1) / TILE : 0;
    }
  }
  const int end = wave_scan(own);
  const uint64_t past = __ballot(end > at);
  if (past == 0) return RowTile{-1, 0, 0};
  const int who = __builtin_ctzll(past);
  int left = at - __builtin_amdgcn_readlane(end - own, who);
  for (int j = 0; j < per; ++j) {
    const int e = who * per + j;
    if (e >= experts) break;
    const int a = max(__builtin_amdgcn_readfirstlane(offsets[e]), 0);
    const int b = min(__builtin_amdgcn_readfirstlane(offsets[e + 1]), rows);
    const int tiles = b > a ? (b - a + TILE - 1) / TILE : 0;
    if (left < tiles) {
      const int r0 = a + left * TILE;
      return RowTile{e, r0, min(r0 + TILE, b)};
    }
    left -= tiles;
  }
  return RowTile{-1, 0, 0};
}

// The row of x that sorted row i takes.
__device__ __forceinline__ int source_row(const RowsArgs& a, int i) {
  if (a.gather == 0) return i;
  const uint32_t o = (uint32_t)a.order[i];
  const int r = (int)(a.gather == 1 ? o : __umulhi(o, a.gather_inv));
  return min(max(r, 0), a.x_rows - 1);
}

// The row of out that sorted row i goes to, -1 for none.
__device__ __forceinline__ int target_row(const RowsArgs& a, int i) {
  if (!a.scatter) return i;
  const int r = a.order[i];
  return (unsigned)r < (unsigned)a.rows ? r : -1;
}

}  // namespace
}  // namespace mxg
