// Products of many MXFP8 rows with FP32 sums (gfx950): mxrows_product and mxmoe_grouped
// of include/mxrows.h. The codes lie in memory and LDS as rows_tile.hip has them; each
// wave takes them and their scales to BF16 in registers (rows_device.h).
//
// A workgroup has a CU alone, and a tile of 128 rows of W by up to 128 of x. Its eight
// waves are two on a SIMD, so that one converts beside the other's products: four waves of
// 64 by 64 take the first 64 of each 128 values of K, four the second, and their sums meet
// in LDS. (Measured alone: a product takes 32 cycles of a SIMD; a wave issues a vector
// instruction every 8 cycles, two one every 4, six of them for a product free. A stage's 16
// products of a wave come with some 100.)
//
// Bound by the matrix cores and what feeds them in the same instruction stream: 1.6 us for
// 256 values of K of a tile, 0.93 with products alone; products, LDS reads and barriers
// 1.1, conversions 0.25, copies 0.2. 4096 rows of 7168 x 8192 434 us in MXFP4 by MXFP8 and 456
// in MXFP8 (1.1 PFLOP/s; a large BF16 product of the library reaches 1.33), 512 rows 59 and
// 65, 203 of 4096 x 16384 41 and 45, 1001 x 2 of 8 experts 4096 x 1024 in MXFP8 37.5.
//
// Left out: four waves, all steps each, alone on a CU (512 rows 84 and 82) or by two (the
// same as this within 7 %, better with many tiles); conversions a stage ahead between the
// products, with and without scheduling groups, the K groups half a stage apart, a higher
// priority for one (all level); a barrier every second stage (level).

#include <hip/hip_runtime.h>

#include "tile_device.h"

namespace mxg {
namespace {

constexpr int kThreads = 512;
constexpr int kRing = 4;  // stages of 128 values of K in LDS

template <int FW>
struct Layout {
  static constexpr int kStepW = FW == MXG_MXFP4 ? 1024 : 2048;
  static constexpr int kWBlock = 2 * kStepW, kXBlock = 32 * 128;  // of 32 rows, a stage
  static constexpr int kX = 4 * kWBlock, kSlot = kX + 4 * kXBlock;
  static constexpr int kScales = kRing * kSlot, kPair = 8 * 256;  // of two stages
  static constexpr int kLds = kScales + kRing / 2 * kPair;
  static constexpr int kSums = 8 * 32 * 256;    // what the waves exchange at the end
  static constexpr int kOutRow = 2 * 64 + 16;   // a row of 64 columns, laid out for the store
  static_assert(kSums + 8 * 32 * kOutRow <= kLds && kLds <= 160 * 1024, "");
};

template <int FW>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
rows_bf16_kernel(RowsArgs a, int row_tiles, int col_tiles, int split) {
  using L = Layout<FW>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave >> 2, ww = wave & 1, wx = wave >> 1 & 1;  // K group; place in the tile
  const int r32 = lane & 31, g = lane >> 5;

  const int at = tile_of_workgroup();
  if (at >= row_tiles * col_tiles * split) return;
  const int tiles = row_tiles * col_tiles;
  const int part = split > 1 ? at / tiles : 0, number = at - part * tiles;
  int ct, rt;
  tile_at(number, row_tiles, col_tiles, &ct, &rt);
  // Rows in blocks of 32, shared evenly among the tiles.
  const int64_t blocks = (a.rows + 31) / 32;
  RowTile tile{0, (int)(32 * (rt * blocks / row_tiles)),
               min((int)(32 * ((rt + 1) * blocks / row_tiles)), a.rows)};
  if (a.offsets) {
    tile = find_tile<128>(a.offsets, a.experts, a.rows, rt, lane);
    if (tile.expert < 0) return;
  }
  const int pair0 = part * a.kp / split, kp = (part + 1) * a.kp / split - pair0;
  const int kbs = min((a.k >> 7) - 2 * pair0, 2 * kp);  // stages that x has

  // The units and scale words of block b of the tile (gated: gate and up blocks in turn).
  const auto block_of = [&](int b) {
    const int rb = a.gated
                       ? min(ct * 2 + (b >> 1), a.nb / 2 - 1) + (b & 1) * (a.nb / 2)
                       : min(ct * 4 + b, a.nb - 1);
    return (int64_t)rb * a.kp + pair0;
  };
  const uint8_t* const we = a.w + tile.expert * a.w_bytes;
  const uint8_t* const wse = a.ws + tile.expert * a.ws_bytes;
  const int64_t base_row = a.gather ? 0 : tile.r0;
  const uint8_t* const xb = a.x + base_row * a.k + (int64_t)pair0 * 256;
  const uint8_t* const xsb = a.xs + base_row * (a.k >> 5) + (int64_t)pair0 * 8;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  // The tile with NX blocks of 32 rows of x for each wave: block t of wave column wx is
  // the tile's block 2 t + wx.
  auto run = [&](auto count) __attribute__((always_inline)) {
    constexpr int NX = decltype(count)::value;
    constexpr int kW = L::kWBlock / 2048;  // KiB of W that a wave copies of a stage
    constexpr int kStage = kW + NX;        // its instructions, without the pair's scales

    // A wave copies half a block of W, NX times 8 rows of x (swizzled: row r holds the 16
    // bytes p of 8 at p ^ r % 8) and, of a pair, the scales of one block of W or x.
    const uint8_t* const wb = we + block_of(wave >> 1) * (2 * L::kWBlock) +
                              (wave & 1) * (L::kWBlock / 2);
    const uint32_t w_to = (wave >> 1) * L::kWBlock + (wave & 1) * (L::kWBlock / 2);
    const int sblock = wave < 4 ? wave : (wave - 4) % (2 * NX);
    int rows[NX + 1];  // of x: those it copies, that of the scales
#pragma unroll
    for (int u = 0; u < NX; ++u) rows[u] = 8 * (wave * NX + u) + (lane >> 3);
    rows[NX] = 32 * sblock + r32;
#pragma unroll
    for (int u = 0; u <= NX; ++u) rows[u] = min(tile.r0 + rows[u], tile.r1 - 1);
    if (a.gather) {  // all entries in one round trip
#pragma unroll
      for (int u = 0; u <= NX; ++u) rows[u] = a.order[rows[u]];
#pragma unroll
      for (int u = 0; u <= NX; ++u) rows[u] = source_of(a, (uint32_t)rows[u]);
    }
    uint32_t xo[NX];
#pragma unroll
    for (int u = 0; u < NX; ++u)
      xo[u] = (uint32_t)(rows[u] - base_row) * (uint32_t)a.k + 16 * ((lane ^ (lane >> 3)) & 7);
    const uint32_t so =
        wave < 4 ? 4 * lane : (uint32_t)(rows[NX] - base_row) * (uint32_t)(a.k >> 5) + 4 * g;
    const uint8_t* const sb = wave < 4 ? wse + block_of(sblock) * 256 : xsb;
    const int s_step = wave < 4 ? 256 : 8;
    const uint32_t s_to = L::kScales + (wave < 4 ? sblock : 4 + sblock) * 256;

    // Past K, where W is zero, x's last stage and scales are taken again.
    auto copy = [&](int j) __attribute__((always_inline)) {
      const uint32_t to = base + (uint32_t)j % kRing * L::kSlot;
      copy_kib<kW>(to + w_to, wb + (int64_t)j * L::kWBlock, 16 * lane);
      const uint8_t* const xj = xb + (int64_t)min(j, kbs - 1) * 128;
#pragma unroll
      for (int u = 0; u < NX; ++u) copy_kib<1>(to + L::kX + 1024 * (wave * NX + u), xj, xo[u]);
      if (j % 2 == 0)
        copy_words(base + s_to + (uint32_t)(j / 2) % (kRing / 2) * L::kPair,
                   sb + (int64_t)(j / 2) * s_step,
                   so - (wave >= 4 && j + 1 >= kbs ? 4 * g : 0));
    };
    const int stages = 2 * kp;
#pragma unroll
    for (int j = 0; j < kRing; ++j)
      if (j < stages) copy(j);

    v16f acc[2][NX];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NX; ++t)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][t][q] = 0.f;

    Piece<FW> pw[2][2];  // operands of a stage and the next
    Piece<MXG_MXFP8> px[2][NX];
    BlockScales sw[2], sx[NX];  // words of a pair: byte S that of step S
    bool check = false;         // whether their bytes may leave BF16's range
    uint32_t again = 0;         // not 0 where a value did
    auto lds16 = [&](uint32_t p) __attribute__((always_inline)) {
      return *reinterpret_cast<const v4u*>(lds + p);
    };
    const uint32_t w_at = 2 * ww * L::kWBlock + kg * L::kStepW + 16 * lane;
    const uint32_t x_at = L::kX + wx * L::kXBlock + 128 * r32 + (16 * (g ^ (r32 & 7)) ^ 64 * kg);
    auto fetch = [&](int j, int set) __attribute__((always_inline)) {
      const uint32_t slot = (uint32_t)j % kRing * L::kSlot;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pw[set][i].lo = lds16(slot + w_at + i * L::kWBlock);
        if constexpr (FW == MXG_MXFP8) pw[set][i].hi = lds16(slot + w_at + i * L::kWBlock + 1024);
      }
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const uint32_t p = slot + 2 * t * L::kXBlock;
        px[set][t].lo = lds16(p + x_at);
        px[set][t].hi = lds16(p + (x_at ^ 32));
      }
    };
    auto fetch_scales = [&](BlockScales (&w)[2], BlockScales (&x)[NX], int pair)
                            __attribute__((always_inline)) {
      const uint8_t* p = lds + L::kScales + (uint32_t)pair % (kRing / 2) * L::kPair + 4 * r32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + (2 * ww + i) * 256);
        w[i] = {q[0], q[32]};
      }
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + (4 + 2 * t + wx) * 256);
        x[t] = {__builtin_amdgcn_perm(q[32], q[0], 0x06040200u),
                __builtin_amdgcn_perm(q[32], q[0], 0x07050301u)};
      }
    };
    auto check_scales = [&]() __attribute__((always_inline)) {
      uint32_t z = ~0u;
#pragma unroll
      for (int i = 0; i < 2; ++i) z &= well_inside(g ? sw[i].second : sw[i].first);
#pragma unroll
      for (int t = 0; t < NX; ++t) z &= well_inside(g ? sx[t].second : sx[t].first);
      check = !__all(all_inside(z));
    };
    // The bytes of the pair's stage `set` in its words.
    auto bytes = [&](const BlockScales& s, int set) __attribute__((always_inline)) {
      const int shift = 8 * (2 * set + kg);
      return BlockScales{s.first >> shift & 0xFFu, s.second >> shift & 0xFFu};
    };
    auto check_values = [&](int set) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) again |= leaves_bf16(by_blocks(pw[set][i]), bytes(sw[i], set));
#pragma unroll
      for (int t = 0; t < NX; ++t) again |= leaves_bf16(px[set][t], bytes(sx[t], set));
    };
    auto contract = [&](int set) __attribute__((always_inline)) {
      Bf16Piece wbf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) wbf[i] = to_bf16(by_blocks(pw[set][i]), bytes(sw[i], set));
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const Bf16Piece xbf = to_bf16(px[set][t], bytes(sx[t], set));
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wbf[i].v[q], xbf.v[q], acc[i][t],
                                                                0, 0, 0);
      }
    };

    // The first stage is there; the others may still fly.
    if (stages >= kRing)
      wait_loads<(kRing - 1) * kStage + kRing / 2 - 1>();
    else
      wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch_scales(sw, sx, 0);
    check_scales();
    fetch(0, 0);
    // Before stage j's products: its operands are in registers (in every wave's, behind the
    // barrier: its slot is free for stage j + kRing), and the next one has to have landed.
    auto next = [&](int j) __attribute__((always_inline)) {
      if (j + kRing <= stages)
        wait_loads<(kRing - 2) * kStage + (kRing - 2) / 2>();
      else
        wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (j + kRing < stages) copy(j + kRing);
    };
    // (A stage's values are looked at, where its pair's scale bytes ask for it, at the end
    // of the one before: between conversions and products the branch cost 0.1 us a stage.)
    if (check) check_values(0);
    for (int pair = 0; pair < kp; ++pair) {
      next(2 * pair);
      fetch(2 * pair + 1, 1);
      contract(0);
      if (check) check_values(1);
      if (pair + 1 < kp) {
        BlockScales nw[2], nx[NX];
        next(2 * pair + 1);
        fetch_scales(nw, nx, pair + 1);
        fetch(2 * pair + 2, 0);
        contract(1);
#pragma unroll
        for (int i = 0; i < 2; ++i) sw[i] = nw[i];
#pragma unroll
        for (int t = 0; t < NX; ++t) sx[t] = nx[t];
        check_scales();
        if (check) check_values(0);
      }
    }
    contract(1);

    if (__any(again != 0)) {
      const uint8_t *wu[2], *xu[NX], *xsu[NX];
      const uint32_t* wsu[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        wu[i] = we + block_of(2 * ww + i) * (2 * L::kWBlock);
        wsu[i] = reinterpret_cast<const uint32_t*>(wse + block_of(2 * ww + i) * 256);
      }
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const int row = source_row(a, min(tile.r0 + 32 * (2 * t + wx) + r32, tile.r1 - 1));
        xu[t] = a.x + (int64_t)row * a.k + (int64_t)pair0 * 256;
        xsu[t] = a.xs + (int64_t)row * (a.k >> 5) + (int64_t)pair0 * 8;
      }
      contract_again<FW>(wu, wsu, xu, xsu, 0, stages, kbs, kg, kg + 1, acc);
    }
#pragma unroll
    for (int t = 0; t < NX; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) asm volatile("s_nop 15\n\ts_nop 15" : "+v"(acc[i][t]));

    // ---- epilogue: K group t has block t of the rows from here on (of one block: group 0)
    int to[4] = {-1, -1, -1, -1};
    const int t = NX == 1 ? 0 : kg;
    const int cols = a.gated ? 32 : 64;  // of the wave
    const int lanes = cols / 8;          // of 16 bytes, for a row
    const bool mine = NX == 2 || kg == 0;
    if (mine && split == 1) {
      int sorted[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        sorted[u] = tile.r0 + 32 * (2 * t + wx) + lane / lanes + u * (64 / lanes);
#pragma unroll
      for (int u = 0; u < 4; ++u) to[u] = min(sorted[u], tile.r1 - 1);
      if (a.scatter) {  // all targets in one round trip
#pragma unroll
        for (int u = 0; u < 4; ++u) to[u] = a.order[to[u]];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (sorted[u] >= tile.r1 || (unsigned)to[u] >= (unsigned)a.rows || u * (64 / lanes) >= 32)
          to[u] = -1;
    }
    __syncthreads();  // (the ring is read out)
    v4f* const sums = reinterpret_cast<v4f*>(lds) + lane;
    auto give = [&](const v16f& v, int i) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sums[((wave ^ 4) * 8 + i * 4 + q) * 64] =
            v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    };
    v16f own[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (NX == 2 && kg == 0) give(acc[i][NX - 1], i);
      if (kg == 1) give(acc[i][0], i);
      own[i] = kg == 0 ? acc[i][0] : acc[i][NX - 1];
    }
    __syncthreads();
    if (!mine) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f v = sums[(wave * 8 + i * 4 + q) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) own[i][4 * q + e] += v[e];
      }
    if (split > 1) {  // sums as they lie, 1 KiB a store, for the join
      v4f* p = reinterpret_cast<v4f*>(a.partial) +
               ((int64_t)(number * split + part) * 4 + (wave & 3)) * 1024 + t * 512 + lane;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[i * 256 + 64 * q] = v4f{own[i][4 * q], own[i][4 * q + 1], own[i][4 * q + 2],
                                    own[i][4 * q + 3]};
      return;
    }
    // 32 rows of the wave's columns meet in LDS and go out by whole lines.
    uint8_t* const out = lds + L::kSums + wave * 32 * L::kOutRow;
    auto lay = [&](const v16f& v, int block) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; q += 2)
        *reinterpret_cast<uint4*>(out + r32 * L::kOutRow + 64 * block + 16 * (q + g)) =
            eight_columns(v, q);
    };
    if (a.gated) {
      lay(gated(own[0], own[1]), 0);
    } else {
      lay(own[0], 0);
      lay(own[1], 1);
    }
    __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
    const int col = ct * 2 * cols + ww * cols + 8 * (lane % lanes);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (to[u] < 0 || col >= a.out_n) continue;
      const v4u v = *reinterpret_cast<const v4u*>(
          out + (lane / lanes + u * (64 / lanes)) * L::kOutRow + 16 * (lane % lanes));
      __builtin_nontemporal_store(
          v, reinterpret_cast<v4u*>(a.out + (int64_t)to[u] * a.out_n + col));
    }
  };
  if (tile.r1 - tile.r0 > 64)
    run(std::integral_constant<int, 2>());
  else
    run(std::integral_constant<int, 1>());
}

}  // namespace

hipError_t launch_rows_bf16(const RowsArgs& a, int w_format, int row_tiles, int col_tiles,
                            int split, hipStream_t s) {
  const TileGrid g = tile_grid((int64_t)row_tiles * col_tiles * split);
  const dim3 grid(g.x, g.y);
  if (w_format == MXG_MXFP4)
    hipLaunchKernelGGL((rows_bf16_kernel<MXG_MXFP4>), grid, dim3(kThreads), 0, s, a,
                       row_tiles, col_tiles, split);
  else
    hipLaunchKernelGGL((rows_bf16_kernel<MXG_MXFP8>), grid, dim3(kThreads), 0, s, a,
                       row_tiles, col_tiles, split);
  return hipGetLastError();
}

}  // namespace mxg
