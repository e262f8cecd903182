// Products of many rows (gfx950): mxrows_product and mxmoe_grouped of
// include/mxrows.h where the matrix cores bound them.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "rows_device.h"

namespace mxg {
namespace {

template <int N>
using Int = std::integral_constant<int, N>;

// 1024 bytes from base + off (a lane's 16) to LDS at `to` (wave-uniform), and
// COUNT - 1 times the next 1024 to the next 1024. The compiler does not see these
// loads: their end is waited for with s_waitcnt vmcnt.
template <int COUNT>
__device__ __forceinline__ void copy_kib(uint32_t to, const uint8_t* base, uint32_t off) {
  static_assert(COUNT == 1 || COUNT == 2 || COUNT == 4, "");
  if constexpr (COUNT == 1)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 ::"s"(to), "v"(off), "s"(base) : "memory");
  else if constexpr (COUNT == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024"
                 ::"s"(to), "v"(off), "s"(base) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:1024\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:2048\n\t"
                 "global_load_lds_dwordx4 %1, %2 offset:3072"
                 ::"s"(to), "v"(off), "s"(base) : "memory");
}
// 256 bytes, 4 a lane.
__device__ __forceinline__ void copy_words(uint32_t to, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(to), "v"(off), "s"(base) : "memory");
}

template <int FW, int FX, int RW, int RX, int WW, int WX>
struct Tile {
  static constexpr int kWaves = WW * WX, kThreads = 64 * kWaves;
  static constexpr int kKb = FX == MXG_MXFP4 ? 2 : 1;  // of a stage: 128 bytes of a row of x
  static constexpr int kSteps = 2 * kKb;
  static constexpr int kWBlock = (FW == MXG_MXFP4 ? 2048 : 4096) * kKb, kXBlock = 4096;
  static constexpr int kNW = WW * RW, kNX = WX * RX;  // blocks of 32 rows
  static constexpr int kRows = 32 * kNX;
  static constexpr int kX = kNW * kWBlock, kWS = kX + kNX * kXBlock, kXS = kWS + kNW * 256;
  static constexpr int kStage = kXS + kNX * 256;
  static constexpr int kCopyW = kNW / kWaves, kCopyX = kNX / kWaves;
  static_assert(kNW % kWaves == 0 && kNX % kWaves == 0 && RW % 2 == 0, "");
};

template <int FW, int FX, int RW, int RX, int WW, int WX>
__global__ void __launch_bounds__(64 * WW * WX) __attribute__((amdgpu_waves_per_eu(1)))
rows_tile_kernel(RowsArgs a, int row_tiles, int col_tiles) {
  using T = Tile<FW, FX, RW, RX, WW, WX>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * T::kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ww = wave % WW, wx = wave / WW;
  const int r32 = lane & 31, g = lane >> 5;

  // Workgroups go to the XCDs in turn: runs of 32 tiles stay on one.
  constexpr int kRun = 32;
  const int bid = blockIdx.x;
  const int at = bid / (8 * kRun) * (8 * kRun) + (bid & 7) * kRun + (bid >> 3) % kRun;
  if (at >= row_tiles * col_tiles) return;
  // Eight row tiles side by side down the columns, so that a run shares W and x.
  constexpr int kGroup = 8;
  const int group = at / (kGroup * col_tiles);
  const int high = min(kGroup, row_tiles - group * kGroup);
  const int in = at - group * kGroup * col_tiles;
  const int ct = in / high, rt = group * kGroup + in % high;
  RowTile tile{0, rt * T::kRows, min(rt * T::kRows + T::kRows, a.rows)};
  if (a.offsets) {
    tile = find_tile<T::kRows>(a.offsets, a.experts, a.rows, rt, lane);
    if (tile.expert < 0) return;
  }

  // ---- what this wave copies ---------------------------------------------------
  const uint8_t *wb[T::kCopyW], *wsb[T::kCopyW];
#pragma unroll
  for (int i = 0; i < T::kCopyW; ++i) {
    const int b = wave + i * T::kWaves;  // of the tile's blocks
    int rb;
    if (a.gated)  // gate and up blocks in turn
      rb = min(ct * (T::kNW / 2) + (b >> 1), a.nb / 2 - 1) + (b & 1) * (a.nb / 2);
    else
      rb = min(ct * T::kNW + b, a.nb - 1);
    wb[i] = a.w + tile.expert * a.w_bytes + (int64_t)rb * a.kp * (FW == MXG_MXFP4 ? 4096 : 8192);
    wsb[i] = a.ws + tile.expert * a.ws_bytes + (int64_t)rb * a.kp * 256;
  }
  // Rows of x: a wave instruction takes 8 rows of 128 bytes, lane l the piece
  // (l ^ l / 8) % 8 of row l / 8, so that a row r holds piece p at p ^ r % 8 and the
  // lanes of an operand read meet no bank twice. Rows past the end: the last one.
  const int x_row = FX == MXG_MXFP4 ? a.k >> 1 : a.k;
  const int64_t base_row = a.gather ? 0 : tile.r0;
  const uint8_t* xb = a.x + base_row * x_row;
  const uint8_t* xsb = a.xs + base_row * (a.k >> 5);
  const int piece = (lane ^ (lane >> 3)) & 7;
  uint32_t xo[T::kCopyX][4], xso[T::kCopyX];
#pragma unroll
  for (int i = 0; i < T::kCopyX; ++i) {
    const int b = wave + i * T::kWaves;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = min(tile.r0 + 32 * b + 8 * j + (lane >> 3), tile.r1 - 1);
      xo[i][j] = (uint32_t)(source_row(a, row) - base_row) * (uint32_t)x_row + 16 * piece;
    }
    const int row = min(tile.r0 + 32 * b + r32, tile.r1 - 1);
    xso[i] = (uint32_t)(source_row(a, row) - base_row) * (uint32_t)(a.k >> 5) +
             (FX == MXG_MXFP4 ? 4 * g : 0);
  }
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int kbs = a.k >> 7;
  const int stages = (kbs + T::kKb - 1) / T::kKb;

  // Copies of a stage, numbered: kCopyW times (codes, scales), kCopyX times (four of
  // codes, scales).
  constexpr int kCopies = 2 * T::kCopyW + 5 * T::kCopyX;
  auto copy = [&](int n, int stage, uint32_t buf) __attribute__((always_inline)) {
    const uint32_t to = base + buf;
    if (n < 2 * T::kCopyW) {
      const int i = n >> 1, b = wave + i * T::kWaves;
      if ((n & 1) == 0)
        copy_kib<T::kWBlock / 1024>(to + b * T::kWBlock, wb[i] + (int64_t)stage * T::kWBlock,
                                    16 * lane);
      else
        copy_words(to + T::kWS + b * 256, wsb[i] + (stage * T::kKb >> 1) * 256, 4 * lane);
    } else {
      const int i = (n - 2 * T::kCopyW) / 5, j = (n - 2 * T::kCopyW) % 5, b = wave + i * T::kWaves;
      // A stage of which K has only the first half: its codes again (W's are zero).
      const bool half = FX == MXG_MXFP4 && 2 * stage + 2 > kbs;
      if (j < 4)
        copy_kib<1>(to + T::kX + b * T::kXBlock + 1024 * j, xb + (int64_t)stage * 128,
                    xo[i][j < 4 ? j : 0] - (half ? 16 * (piece & 4) : 0));
      else
        copy_words(to + T::kXS + b * 256, xsb + stage * 4 * T::kKb, xso[i] - (half ? 4 * g : 0));
    }
  };

  // ---- what it computes -----------------------------------------------------------
  v16f acc[RW][RX];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int t = 0; t < RX; ++t)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][t][q] = 0.f;
  struct Operands {
    Piece<FW> w[RW];
    Piece<FX> x[RX];
  } op[2];
  uint32_t sw[RW], sx[RX];

  const uint32_t w_at = ww * RW * T::kWBlock + 16 * lane;
  const uint32_t x_at = T::kX + wx * RX * T::kXBlock + 128 * r32 +
                        16 * ((FX == MXG_MXFP4 ? 2 * g : g) ^ (r32 & 7));
  auto lds16 = [&](uint32_t at) __attribute__((always_inline)) {
    return *reinterpret_cast<const v4u*>(lds + at);
  };
  // The n-th operand of a step: W's, then x's. buf: the buffer's offset.
  auto fetch = [&](Operands& o, int n, auto step, uint32_t buf) __attribute__((always_inline)) {
    constexpr int S = decltype(step)::value;
    if (n < RW) {
      const uint32_t p = buf + w_at + n * T::kWBlock + S * (FW == MXG_MXFP4 ? 1024 : 2048);
      o.w[n].lo = lds16(p);
      if constexpr (FW == MXG_MXFP8) o.w[n].hi = lds16(p + 1024);
    } else {
      const int t = n - RW;
      if constexpr (FX == MXG_MXFP4) {
        o.x[t].lo = lds16(buf + t * T::kXBlock + (x_at ^ (16 * (4 * (S >> 1) + (S & 1)))));
      } else {
        o.x[t].lo = lds16(buf + t * T::kXBlock + (x_at ^ (32 * S)));
        o.x[t].hi = lds16(buf + t * T::kXBlock + (x_at ^ (64 + 32 * S)));
      }
    }
  };
  // A stage's scales, byte S of a word that of step S.
  auto fetch_scales = [&](uint32_t (&w)[RW], uint32_t (&x)[RX], int stage, uint32_t buf)
                          __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      w[i] = *reinterpret_cast<const uint32_t*>(lds + buf + T::kWS + (ww * RW + i) * 256 + 4 * lane);
      if constexpr (FX == MXG_MXFP8) w[i] >>= 16 * (stage & 1);
    }
#pragma unroll
    for (int t = 0; t < RX; ++t) {
      const uint8_t* p = lds + buf + T::kXS + (wx * RX + t) * 256 + 4 * r32;
      const uint32_t d0 = *reinterpret_cast<const uint32_t*>(p);
      if constexpr (FX == MXG_MXFP4) {
        const uint32_t d1 = *reinterpret_cast<const uint32_t*>(p + 128);
        x[t] = __builtin_amdgcn_perm(d1, d0, g ? 0x07060302u : 0x05040100u);
      } else {
        x[t] = d0 >> (16 * g);
      }
    }
  };

  // One step of stage `stage` in the buffer at buf: its products, between them the
  // next step's operands (kNext) and, in a stage's last one, the copies of the stage
  // after the next (kCopy).
  auto step = [&](auto number, auto next, auto copies, int stage, uint32_t buf)
                  __attribute__((always_inline)) {
    constexpr int S = decltype(number)::value, kM = RW * RX, kCur = S & 1;
    constexpr bool kLast = S == T::kSteps - 1;
    constexpr bool kNext = !kLast || decltype(next)::value, kCopy = kLast && decltype(copies)::value;
    const uint32_t other = T::kStage - buf;
    uint32_t nw[RW], nx[RX];
    if constexpr (kLast && kNext) {
      // The next stage has landed, every wave is done reading this one.
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      fetch_scales(nw, nx, stage + 1, other);
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int i = m % RW, t = m / RW;
      acc[i][t] = product<FW, FX, S, S>(op[kCur].w[i], sw[i], op[kCur].x[t], sx[t], acc[i][t]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kNext) {
#pragma unroll
        for (int n = m * (RW + RX) / kM; n < (m + 1) * (RW + RX) / kM; ++n)
          fetch(op[kCur ^ 1], n, Int<kLast ? 0 : S + 1>(), kLast ? other : buf);
      }
      if constexpr (kCopy) {
#pragma unroll
        for (int n = m * kCopies / kM; n < (m + 1) * kCopies / kM; ++n) copy(n, stage + 2, buf);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kLast && kNext) {
#pragma unroll
      for (int i = 0; i < RW; ++i) sw[i] = nw[i];
#pragma unroll
      for (int t = 0; t < RX; ++t) sx[t] = nx[t];
    }
  };
  auto whole = [&](auto next, auto copies, int stage, uint32_t buf) __attribute__((always_inline)) {
    step(Int<0>(), next, copies, stage, buf);
    step(Int<1>(), next, copies, stage, buf);
    if constexpr (T::kSteps == 4) {
      step(Int<2>(), next, copies, stage, buf);
      step(Int<3>(), next, copies, stage, buf);
    }
  };

#pragma unroll
  for (int n = 0; n < kCopies; ++n) copy(n, 0, 0);
  if (stages > 1) {
#pragma unroll
    for (int n = 0; n < kCopies; ++n) copy(n, 1, T::kStage);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  fetch_scales(sw, sx, 0, 0);
#pragma unroll
  for (int n = 0; n < RW + RX; ++n) fetch(op[0], n, Int<0>(), 0);
  uint32_t buf = 0;
  int s = 0;
  for (; s + 2 < stages; ++s) {
    whole(Int<1>(), Int<1>(), s, buf);
    buf = T::kStage - buf;
  }
  if (stages > 1) {
    whole(Int<1>(), Int<0>(), s, buf);
    buf = T::kStage - buf;
    ++s;
  }
  whole(Int<0>(), Int<0>(), s, buf);

  // ---- epilogue ---------------------------------------------------------------------
  // A lane's four neighbouring columns meet those of the lane 32 on: 16 bytes.
#pragma unroll
  for (int t = 0; t < RX; ++t) {
    const int i0 = tile.r0 + 32 * (wx * RX + t) + r32;
    const int to = i0 < tile.r1 ? target_row(a, i0) : -1;
    uint16_t* row = a.out + (int64_t)max(to, 0) * a.out_n;
    auto store = [&](const v16f& v, int col) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const auto lo = __builtin_amdgcn_permlane32_swap(bf16_pair(v[4 * q], v[4 * q + 1]),
                                                         bf16_pair(v[4 * q + 4], v[4 * q + 5]),
                                                         false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(bf16_pair(v[4 * q + 2], v[4 * q + 3]),
                                                         bf16_pair(v[4 * q + 6], v[4 * q + 7]),
                                                         false, false);
        const int c = col + 8 * (q + g);
        if (to >= 0 && c < a.out_n)
          *reinterpret_cast<uint4*>(row + c) = uint4{lo[0], hi[0], lo[1], hi[1]};
      }
    };
    if (a.gated) {
#pragma unroll
      for (int i = 0; i < RW; i += 2) {
        v16f h;
#pragma unroll
        for (int q = 0; q < 16; ++q) h[q] = gated(acc[i][t][q], acc[i + 1][t][q]);
        store(h, 32 * (ct * (T::kNW / 2) + (ww * RW + i) / 2));
      }
    } else {
#pragma unroll
      for (int i = 0; i < RW; ++i) store(acc[i][t], 32 * (ct * T::kNW + ww * RW + i));
    }
  }
}

template <int FW, int FX, int RW, int RX, int WW, int WX>
hipError_t launch(const RowsArgs& a, hipStream_t s) {
  using T = Tile<FW, FX, RW, RX, WW, WX>;
  const int64_t most = a.rows / T::kRows + (a.experts < a.rows ? a.experts : a.rows);
  const int64_t rt = a.offsets ? most : (a.rows + T::kRows - 1) / T::kRows;
  const int64_t ct = (a.nb + T::kNW - 1) / T::kNW;
  const int64_t grid = (rt * ct + 255) / 256 * 256;
  if (grid * T::kThreads > UINT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((rows_tile_kernel<FW, FX, RW, RX, WW, WX>), dim3((unsigned)grid),
                     dim3(T::kThreads), 0, s, a, (int)rt, (int)ct);
  return hipGetLastError();
}

template <int FW, int FX>
hipError_t by_size(const RowsArgs& a, hipStream_t s) {
  return launch<FW, FX, 4, 4, 2, 2>(a, s);
}

}  // namespace

hipError_t launch_rows_tile(const RowsArgs& a, int w_format, int x_format, hipStream_t s) {
  if (x_format == MXG_MXFP4) return by_size<MXG_MXFP4, MXG_MXFP4>(a, s);
  if (w_format == MXG_MXFP4) return by_size<MXG_MXFP4, MXG_MXFP8>(a, s);
  return by_size<MXG_MXFP8, MXG_MXFP8>(a, s);
}

}  // namespace mxg
