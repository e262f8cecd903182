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

// ---- MXFP8 in BF16 -------------------------------------------------------------
//
// The scaled MFMA drops what lies 2^-13 below the largest of eight neighbouring
// products as soon as one side is MXFP8. So that FP32 sums keep it, the operands go to
// BF16 with their scales and through v_mfma_f32_32x32x16_bf16, four for a step of 64,
// from the same registers: an operand's `lo` lies in the step's first block of 32
// values, its `hi` in the second (16 values on from 16 (l / 32) of each). An E2M1 or
// e4m3 value times 2^(s-127) is a BF16 value for every scale byte s of 3..246. The main
// loops take all of them so, note whether one was not (leaves_bf16), and contract_again
// redoes a wave's sums then.

// MXFP4's 16 values of a lane lie in one block: halves change places between the lane
// groups. MXFP8's lie in both already.
__device__ __forceinline__ Piece<MXG_MXFP8> by_blocks(const Piece<MXG_MXFP8>& p) { return p; }
__device__ __forceinline__ Piece<MXG_MXFP4> by_blocks(const Piece<MXG_MXFP4>& p) {
  const auto a = __builtin_amdgcn_permlane32_swap(p.lo.x, p.lo.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(p.lo.y, p.lo.w, false, false);
  return {v4u{a[0], b[0], a[1], b[1]}};
}

__device__ __forceinline__ v8bf fp4x8_to_bf16(uint32_t w, float scale) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The scale bytes of a row's two blocks of a step.
struct BlockScales {
  uint32_t first, second;
};
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// A step's operand in BF16, of a piece by blocks.
struct Bf16Piece {
  v8bf v[4];
};
__device__ __forceinline__ Bf16Piece to_bf16(const Piece<MXG_MXFP8>& p, const BlockScales& s) {
  const float a = scale_of(s.first), b = scale_of(s.second);
  return {{fp8x8_to_bf16(p.lo.x, p.lo.y, a), fp8x8_to_bf16(p.lo.z, p.lo.w, a),
           fp8x8_to_bf16(p.hi.x, p.hi.y, b), fp8x8_to_bf16(p.hi.z, p.hi.w, b)}};
}
__device__ __forceinline__ Bf16Piece to_bf16(const Piece<MXG_MXFP4>& p, const BlockScales& s) {
  const float a = scale_of(s.first), b = scale_of(s.second);
  return {{fp4x8_to_bf16(p.lo.x, a), fp4x8_to_bf16(p.lo.y, a), fp4x8_to_bf16(p.lo.z, b),
           fp4x8_to_bf16(p.lo.w, b)}};
}

__device__ __forceinline__ v16f product(const Bf16Piece& w, const Bf16Piece& x, v16f acc) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w.v[j], x.v[j], acc, 0, 0, 0);
  return acc;
}

// Bit 7 of every byte set that lies in 64..191: well inside 3..246, where the scale
// bytes of ordinary tensors are, and asked in two instructions.
__device__ __forceinline__ uint32_t well_inside(uint32_t w) { return w ^ (w << 1); }
__device__ __forceinline__ bool all_inside(uint32_t z) { return (~z & 0x80808080u) == 0; }

// Not 0 where BF16 may not hold the values of a lane's piece by blocks: a scale byte
// outside 3..246 with a nonzero code beside it (a block of zeros quantizes to scale
// byte 0), or the NaN 255. (Without branches: the main loops ask in one.)
__device__ __forceinline__ uint32_t leaves_bf16(uint32_t scale, uint32_t codes) {
  return scale - 3u > 243u ? codes | (scale == 0xFFu) : 0u;
}
__device__ __forceinline__ uint32_t leaves_bf16(const Piece<MXG_MXFP8>& p, const BlockScales& s) {
  return leaves_bf16(s.first, (p.lo.x | p.lo.y | p.lo.z | p.lo.w) & 0x7F7F7F7Fu) |
         leaves_bf16(s.second, (p.hi.x | p.hi.y | p.hi.z | p.hi.w) & 0x7F7F7F7Fu);
}
__device__ __forceinline__ uint32_t leaves_bf16(const Piece<MXG_MXFP4>& p, const BlockScales& s) {
  return leaves_bf16(s.first, (p.lo.x | p.lo.y) & 0x77777777u) |
         leaves_bf16(s.second, (p.lo.z | p.lo.w) & 0x77777777u);
}

// The sums of RW by NX blocks of 32 rows once more, from memory, steps s0..s1-1 of the
// kb's from kb0 to kb1-1: in BF16, and by the scaled instruction where BF16 does not hold
// a value. w, ws: a block's units and scale words; x, xs: a lane's row. kbs: the kb's
// there are (past them W is zero, and x's last one is taken again).
template <int FW, int RW, int NX>
__device__ __forceinline__ void contract_again(const uint8_t* const (&w)[RW],
                                               const uint32_t* const (&ws)[RW],
                                               const uint8_t* const (&x)[NX],
                                               const uint8_t* const (&xs)[NX], int kb0, int kb1,
                                               int kbs, int s0, int s1, v16f (&acc)[RW][NX]) {
  constexpr int kStep = FW == MXG_MXFP4 ? 1024 : 2048;
  const int lane = threadIdx.x & 63, r32 = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int t = 0; t < NX; ++t)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][t][q] = 0.f;
#pragma unroll 1
  for (int kb = kb0; kb < kb1; ++kb) {
    const int xkb = min(kb, kbs - 1);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      Piece<FW> pw[RW];
      Piece<MXG_MXFP8> px[NX];
      BlockScales sw[RW], sx[NX];
      uint32_t leaves = 0;
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const uint8_t* u = w[i] + (int64_t)(2 * kb + s) * kStep + 16 * lane;
        pw[i].lo = *reinterpret_cast<const v4u*>(u);
        if constexpr (FW == MXG_MXFP8) pw[i].hi = *reinterpret_cast<const v4u*>(u + 1024);
        const uint32_t* q = ws[i] + (kb >> 1) * 64 + r32;
        const int shift = 8 * (2 * (kb & 1) + s);
        sw[i] = {q[0] >> shift & 0xFFu, q[32] >> shift & 0xFFu};
        leaves |= leaves_bf16(by_blocks(pw[i]), sw[i]);
      }
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const uint8_t* u = x[t] + 128 * xkb + 64 * s + 16 * g;
        px[t].lo = *reinterpret_cast<const v4u*>(u);
        px[t].hi = *reinterpret_cast<const v4u*>(u + 32);
        const uint32_t q = *reinterpret_cast<const uint32_t*>(xs[t] + 4 * xkb);
        sx[t] = {q >> (16 * s) & 0xFFu, q >> (16 * s + 8) & 0xFFu};
        leaves |= leaves_bf16(px[t], sx[t]);
      }
      if (__any(leaves != 0)) {
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
          for (int t = 0; t < NX; ++t)
            acc[i][t] = product<FW, MXG_MXFP8, 0, 0>(pw[i], g ? sw[i].second : sw[i].first, px[t],
                                                     g ? sx[t].second : sx[t].first, acc[i][t]);
      } else {
#pragma unroll
        for (int t = 0; t < NX; ++t) {
          const Bf16Piece xb = to_bf16(px[t], sx[t]);
#pragma unroll
          for (int i = 0; i < RW; ++i)
            acc[i][t] = product(to_bf16(by_blocks(pw[i]), sw[i]), xb, acc[i][t]);
        }
      }
    }
  }
}

// silu(gate) * up. With E = exp(-|gate|), silu is gate / (1 + E) for a gate from zero
// on and gate E / (1 + E) below: the reciprocal's argument lies in 1..2. E is q^3 of q =
// exp2(-|gate| log2(e) / 3), and its factors join the product one by one: E and silu
// leave FP32's normal range from gates of -87 and -91 on, their product with a large up
// does not (q does at -262, where E is below 2^-377). No partial product overflows
// where the whole does not: |gate| q / 2 / (1 + E) stays below 0.53, and 2 q follows. E is
// off by |gate| 2^-23 and a few 2^-24 of itself (the exponent's rounding), far below the
// result's BF16 rounding; expf and a division took twice the time of a tile's epilogue.
__device__ __forceinline__ float gated(float gate, float up) {
  const float q = __builtin_amdgcn_exp2f(fabsf(gate) * -0.48089835f);
  const float f = gate < 0.f ? q : 1.f;
  const float s = gate * f * (0.5f * __builtin_amdgcn_rcpf(1.f + q * q * q));
  return s * up * (2.f * f) * f;
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

// The row of x that an entry of the order leads to.
__device__ __forceinline__ int source_of(const RowsArgs& a, uint32_t o) {
  const int r = (int)(a.gather == 1 ? o : over_gather(o, a.over));
  return min(max(r, 0), a.x_rows - 1);
}

// The row of x that sorted row i takes.
__device__ __forceinline__ int source_row(const RowsArgs& a, int i) {
  return a.gather == 0 ? i : source_of(a, (uint32_t)a.order[i]);
}

// The row of out that sorted row i goes to, -1 for none.
__device__ __forceinline__ int target_row(const RowsArgs& a, int i) {
  if (!a.scatter) return i;
  const int r = a.order[i];
  return (unsigned)r < (unsigned)a.rows ? r : -1;
}

}  // namespace
}  // namespace mxg
