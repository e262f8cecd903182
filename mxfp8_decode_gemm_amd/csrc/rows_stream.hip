// Products of few rows (gfx950): mxrows_product and mxmoe_grouped of
// include/mxrows.h where a weight is read for at most a few dozen rows (the sums of
// rows_tile.hip, on the same instruction).
//
// What bounds it: the read of the active weights. A workgroup takes 32 rows of W
// (gated: 32 gate rows and the up rows beside them) and up to 32 rows of x; its eight
// waves divide K, so that even a narrow weight has many waves reading. Each wave
// streams its units (1 KiB contiguous per instruction) and the rows' codes (in
// L2) into registers and feeds both to the scaled MFMA as they are; the partial
// tiles meet in LDS and are summed in ascending K order.
//
// MXFP8 rows go through BF16 (BF; rows_device.h) unless they are to be fast.
//
// One row of 7168 x 8192 in MXFP4 7.7 us (31 MB, 4.1 TB/s; a wave asks for the next 256 of K
// when it has multiplied the last), 8 in MXFP8 13.0 us (4.7 TB/s; fast 14.4); 8 tokens x 8 of
// 64 experts of 4096 x 7168 gated, MXFP4 by MXFP8, 96 to 108 us (656 MB, 6.1 to 6.8 TB/s; fast
// 101). Left out: units in a register ring of 2 to 6 (experts slower, one weight level), 16
// waves, 64 rows of x.

#include <hip/hip_runtime.h>

#include "rows_device.h"

namespace mxg {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// BF: MXFP8 contracted in BF16 (rows_device.h).
template <int FW, int FX, bool GATED, bool BF>
__global__ void __launch_bounds__(kThreads, 4) rows_stream_kernel(RowsArgs a) {
  constexpr int RW = GATED ? 2 : 1;
  constexpr int kTile = 32;
  __shared__ float red[kWaves][RW][16][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, g = lane >> 5;
  const int ct = blockIdx.y, rt = blockIdx.x;
  RowTile tile{0, rt * kTile, min(rt * kTile + kTile, a.rows)};
  if (a.offsets) {
    tile = find_tile<kTile>(a.offsets, a.experts, a.rows, rt, lane);
    if (tile.expert < 0) return;
  }

  // This lane's row of x (past the end: the last one again).
  const int x_row = FX == MXG_MXFP4 ? a.k / 2 : a.k;
  const int64_t row = source_row(a, min(tile.r0 + r32, tile.r1 - 1));
  const uint8_t* xr = a.x + row * x_row;
  const uint8_t* xsr = a.xs + row * (a.k >> 5);
  constexpr int kUnit = FW == MXG_MXFP4 ? 2048 : 4096;
  const uint8_t* w[RW];
  const uint32_t* ws[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int rb = ct + i * (a.nb / 2);
    w[i] = a.w + tile.expert * a.w_bytes + (int64_t)rb * a.kp * 2 * kUnit + 16 * lane;
    ws[i] = reinterpret_cast<const uint32_t*>(a.ws + tile.expert * a.ws_bytes) +
            (int64_t)rb * a.kp * 64 + lane;
  }

  v16f acc[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i][q] = 0.f;

  uint32_t again = 0;  // (BF) not 0 where BF16 did not hold a value
  const int kbs = a.k >> 7;
  const int p0 = wave * a.kp / kWaves, p1 = (wave + 1) * a.kp / kWaves;
  for (int p = p0; p < p1; ++p) {
    uint32_t sw[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) sw[i] = ws[i][p * 64];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // A kb past K (the packed codes there are zeros): the row's last one again.
      const int kb = min(2 * p + h, kbs - 1);
      Piece<FX> xp[2];
      Piece<FW> wp[RW][2];
      const uint32_t sx = *reinterpret_cast<const uint32_t*>(xsr + 4 * kb);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if constexpr (FX == MXG_MXFP4) {
          xp[s].lo = *reinterpret_cast<const v4u*>(xr + 64 * kb + 16 * (2 * s + g));
        } else {
          xp[s].lo = *reinterpret_cast<const v4u*>(xr + 128 * kb + 64 * s + 16 * g);
          xp[s].hi = *reinterpret_cast<const v4u*>(xr + 128 * kb + 64 * s + 32 + 16 * g);
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const uint8_t* u = w[i] + (int64_t)(2 * p + h) * kUnit;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if constexpr (FW == MXG_MXFP4) {
            wp[i][s].lo = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(u + 1024 * s));
          } else {
            wp[i][s].lo = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(u + 2048 * s));
            wp[i][s].hi =
                __builtin_nontemporal_load(reinterpret_cast<const v4u*>(u + 2048 * s + 1024));
          }
        }
      }
      if constexpr (BF) {
        uint32_t z = well_inside(sx);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const uint32_t inside = well_inside(sw[i]);
          z &= h ? inside | 0x8080u : inside | 0x80800000u;
        }
        const bool check = !__all(all_inside(z));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const BlockScales xs = {sx >> (16 * s) & 0xFFu, sx >> (16 * s + 8) & 0xFFu};
          if (check) again |= leaves_bf16(xp[s], xs);
          const Bf16Piece xb = to_bf16(xp[s], xs);
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const auto both = __builtin_amdgcn_permlane32_swap(sw[i], sw[i], false, false);
            const int shift = 8 * (2 * h + s);
            const BlockScales w = {both[0] >> shift & 0xFFu, both[1] >> shift & 0xFFu};
            const Piece<FW> p = by_blocks(wp[i][s]);
            if (check) again |= leaves_bf16(p, w);
            acc[i] = product(to_bf16(p, w), xb, acc[i]);
            // (One operand of W after the other: two workgroups' registers on a CU.)
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          // (Shifted here, after the loads have been issued.)
          const uint32_t s = h ? sw[i] >> 16 : sw[i], x = sx >> (8 * g);
          acc[i] = product<FW, FX, 0, 0>(wp[i][0], s, xp[0], x, acc[i]);
          acc[i] = product<FW, FX, 1, 2>(wp[i][1], s, xp[1], x, acc[i]);
        }
      }
    }
  }

  if constexpr (BF) {
    if (__any(again != 0)) {
      const uint8_t *wu[RW], *xu[1] = {xr}, *xsu[1] = {xsr};
      const uint32_t* wsu[RW];
      v16f sums[RW][1];
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        wu[i] = w[i] - 16 * lane;
        wsu[i] = ws[i] - lane;
      }
      contract_again<FW>(wu, wsu, xu, xsu, 2 * p0, 2 * p1, kbs, 0, 2, sums);
#pragma unroll
      for (int i = 0; i < RW; ++i) acc[i] = sums[i][0];
    }
  }

  // The sums are read no sooner than the last products have ended.
#pragma unroll
  for (int i = 0; i < RW; ++i) asm volatile("s_nop 15\n\ts_nop 15" : "+v"(acc[i]));
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) red[wave][i][q][lane] = acc[i][q];
  __syncthreads();
  // One thread per row and pair of neighbouring columns.
  for (int u = tid; u < kTile * 16; u += kThreads) {
    const int row = u % kTile, c = 2 * (u / kTile);
    const int l = row + 32 * ((c >> 2) & 1), q = 4 * (c >> 3) + (c & 3);
    if (tile.r0 + row >= tile.r1 || 32 * ct + c >= a.out_n) continue;
    const int to = target_row(a, tile.r0 + row);
    if (to < 0) continue;
    float v[RW][2] = {};
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        v[i][0] += red[k][i][q][l];
        v[i][1] += red[k][i][q + 1][l];
      }
    if constexpr (GATED) {
      v[0][0] = gated(v[0][0], v[1][0]);
      v[0][1] = gated(v[0][1], v[1][1]);
    }
    *reinterpret_cast<uint32_t*>(a.out + (int64_t)to * a.out_n + 32 * ct + c) =
        bf16_pair(v[0][0], v[0][1]);
  }
}

template <int FW, int FX, bool BF>
hipError_t launch(const RowsArgs& a, hipStream_t s) {
  const int64_t most = a.rows / 32 + (a.experts < a.rows ? a.experts : a.rows);
  const dim3 grid((unsigned)(a.offsets ? most : (a.rows + 31) / 32),
                  (unsigned)(a.gated ? a.nb / 2 : a.nb));
  if (a.gated)
    hipLaunchKernelGGL((rows_stream_kernel<FW, FX, true, BF>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((rows_stream_kernel<FW, FX, false, BF>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_stream(const RowsArgs& a, int w_format, int x_format, hipStream_t s) {
  if (x_format == MXG_MXFP4) return launch<MXG_MXFP4, MXG_MXFP4, false>(a, s);
  if (w_format == MXG_MXFP4)
    return a.fast ? launch<MXG_MXFP4, MXG_MXFP8, false>(a, s)
                  : launch<MXG_MXFP4, MXG_MXFP8, true>(a, s);
  return a.fast ? launch<MXG_MXFP8, MXG_MXFP8, false>(a, s)
                : launch<MXG_MXFP8, MXG_MXFP8, true>(a, s);
}

}  // namespace mxg
