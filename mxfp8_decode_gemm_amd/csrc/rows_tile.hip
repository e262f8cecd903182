// Products of many rows (gfx950): mxrows_product and mxmoe_grouped of
// include/mxrows.h where the matrix cores bound them, of MXFP4 rows and of MXFP8 rows that are
// to be fast (rows_bf16.hip takes the others).
//
//   y[r][n] = sum over blocks b of 32 of 2^(sw[n][b] + sx[r][b] - 254) sum of w[n][.] x[r][.]
//
// on v_mfma_scale_f32_32x32x64_f8f6f4, W's rows as its A, x's as its B, so that a lane
// holds neighbouring columns of a row of y. W lies in global memory as the instruction's
// lanes take it (rows_internal.h) and goes to LDS by whole KiB; x goes there by rows,
// swizzled. Both are copied without registers in between, stages ahead of the products,
// behind one barrier and one wait a stage; operands come to registers one step ahead; sums
// stay in the accumulators. FP32 sums, rounded once, at the end. The wait counts the loads
// that may still fly, but small tiles by two with equal formats have a ring of two stages
// and wait for all. In the tiles of 256, which hold every register of a SIMD, four words of
// a lane's addresses lie in scratch; one comes back right behind the wait for the first
// stage, and its own wait is for all the stages copied by then.
//
// A tile is 256 rows of W by up to 256 of x, one workgroup with all of a CU's registers,
// where there are enough of them (4096 rows of 7168 x 8192 in MXFP4 124 us, 3.9 PFLOP/s;
// 4096 tokens x 8 of 64 experts of 4096 x 7168 gated 620 us, 3.1 PFLOP/s with the ends of
// groups counted as work done for nothing). That is bound by power: random MXFP4 operands
// let the matrix cores run at 7.4 PFLOP/s at 1.80 GHz with nothing else; here the products
// alone take 44 us of 56 (4096 x 4096 x 8192), 47 with the operand reads, 52 with the
// copies instead, and the clock falls to 1.5 GHz (without products 37 us at 2.15 GHz). Per
// workgroup 3.5 us before the first product (5.8 with an order) and 5 to 6 us of results:
// an order's entries are loaded one after the other, 3 to 6 of x's rows before the first
// copy, and with results that go by it 16 or 32 of theirs behind the last product (4096 x 8
// rows of 64 experts of 7168 x 2048 in MXFP4 403 us in place, 463 scattered).
//
// Else a tile is 128 by 128, on a CU alone or by two, K divided where too few (512 rows of
// 7168 x 8192 26 us in MXFP4; fast, 203 of 4096 x 16384 in MXFP4 by MXFP8 20 us and 4 to add
// up, 512 of 7168 x 8192 in MXFP8 44). Those are bound by copies out of L2, 32 KiB for 128 x
// 128 x 256 products in MXFP4, and by their starts and ends.
//
// Left out: 128-row tiles for large problems (rows_choice.h), tiles of 128 x 256 with a divided
// K (level), copies past the caches (52 -> 60 us), XCD runs of 16 or 64 tiles and groups
// of 4 or 16 row tiles (within 2 %).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "tile_device.h"

namespace mxg {
namespace {

template <int N>
using Int = std::integral_constant<int, N>;

// A tile's geometry. A stage is kLine bytes of each row of x (of 64: 128 values in MXFP4,
// two MFMA steps, 64 in MXFP8, one) with the same K of W; a ring of them lies in LDS.
// Scales come by pairs of kb (four steps).
// RX: the most 32-row blocks of x of a wave; a tile of fewer rows runs with fewer.
template <int FW, int FX, int RW, int RX, int WW, int WX, bool DEEP>
struct Tile {
  static constexpr int kWaves = WW * WX, kThreads = 64 * kWaves;
  // Bytes of a row of x in a stage. A CU copies whole lines of 128 bytes out of L2 at 125
  // bytes a ns, halves at 72: that bounds a small tile (203 rows of 4096 x 16384 in MXFP4
  // by MXFP8, fast, 27 us with whole lines, 31 with halves). A large one reads less of x for its
  // products and is as fast with halves, of which a ring holds more stages.
  static constexpr int kLine = RX == 2 ? 128 : 64;
  static constexpr int kPer = kLine / (FX == MXG_MXFP4 ? 32 : 64);  // steps of a stage
  static constexpr int kStages = 4 / kPer;              // of a pair
  static constexpr int kStepW = FW == MXG_MXFP4 ? 1024 : 2048;
  static constexpr int kWBlock = kStepW * kPer, kXBlock = 32 * kLine;
  static constexpr int kNW = WW * RW, kNX = WX * RX;  // blocks of 32 rows
  static constexpr int kRows = 32 * kNX;
  static constexpr int kX = kNW * kWBlock, kSlot = kX + kNX * kXBlock;
  // Slots, and stages copied ahead. A large tile: four slots against three 125 us and 128
  // (4096 rows of 7168 x 8192 in MXFP4); ahead by three, since by four is level and starts
  // later (4096 rows of 7168 x 4096 68.3 and 69.0). Small ones share a CU's LDS by two, or
  // where there is one for each CU have it alone, twice as deep (512 rows of 7168 x 8192
  // 44 us in MXFP8 and 26 in MXFP4, 62 and 36 with half the ring; two on a CU by half
  // rings of whole lines against four slots of half lines 392 us and 418, 64 experts of
  // 4096 x 7168 in MXFP8 gated with 64 rows each).
  static constexpr int kRing = RX == 8 ? 4 : (FW == FX ? 2 : 3) * (DEEP ? 2 : 1);
  static constexpr int kAhead = RX == 8 ? 3 : kRing;
  // Pairs that the stages ahead reach into; the ring of scales holds theirs.
  static constexpr int kLefts = (kAhead + kStages - 1) / kStages;
  static constexpr int kScaleRing = kLefts <= 2 ? 2 : 4;
  static constexpr int kXLoads = kLine / 32;  // instructions for a block of x
  static constexpr int kScales = kRing * kSlot, kPair = (kNW + kNX) * 256;
  static constexpr int kLds = kScales + kScaleRing * kPair;
  static constexpr int kCopyW = kNW / kWaves;  // blocks that a wave copies
  static constexpr bool kSplits = RX == 2;     // K may be divided among workgroups
  // Workgroups of a CU (by registers and LDS).
  static constexpr int kResident = RX == 8 || DEEP ? 1 : 2;
  // Instructions of a wave's copies of the stages from..to-1 with `copy_x` blocks of x
  // each; a pair's scales go with its first stage. And of the first 1 / kPer of a
  // stage's copies.
  static constexpr int scales(int stage, int copy_x) {
    return stage % kStages == 0 ? kCopyW + copy_x : 0;
  }
  static constexpr int loads(int from, int to, int copy_x) {
    int n = 0;
    for (int q = from; q < to; ++q)
      n += kCopyW * (kWBlock / 1024) + kXLoads * copy_x + scales(q, copy_x);
    return n;
  }
  static constexpr int first_half(int stage, int copy_x) {
    const int all = kCopyW + kXLoads * copy_x + scales(stage, copy_x);
    int n = 0;
    for (int c = 0; c < all / kPer; ++c) n += c < kCopyW ? kWBlock / 1024 : 1;
    return n;
  }
  // What the epilogue lays out at once: 32 rows of a wave's columns, a row's 16 bytes
  // longer than they are, so that eight rows meet no bank twice.
  static constexpr int kOutRow = 64 * RW + 16;
  static_assert(kNW % kWaves == 0 && RW % 2 == 0 && kResident * kLds <= 160 * 1024, "");
  static_assert(kWaves * 32 * kOutRow <= kScales, "");
};

template <int FW, int FX, int RW, int RX, int WW, int WX, bool DEEP>
__global__ void __launch_bounds__(64 * WW * WX)
__attribute__((amdgpu_waves_per_eu(Tile<FW, FX, RW, RX, WW, WX, DEEP>::kResident)))
rows_tile_kernel(RowsArgs a, int row_tiles, int col_tiles, int split) {
  using T = Tile<FW, FX, RW, RX, WW, WX, DEEP>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ww = wave % WW, wx = wave / WW;
  const int r32 = lane & 31, g = lane >> 5;

  const int at = tile_of_workgroup();
  if (at >= row_tiles * col_tiles * split) return;
  // The tiles of one part of K after the other: those of a run share its rows of x.
  const int tiles = row_tiles * col_tiles;
  const int part = split > 1 ? at / tiles : 0, number = at - part * tiles;
  int ct, rt;
  tile_at(number, row_tiles, col_tiles, &ct, &rt);
  // Rows in blocks of 32, shared evenly among the tiles.
  const int64_t blocks = (a.rows + 31) / 32;
  RowTile tile{0, (int)(32 * (rt * blocks / row_tiles)),
               min((int)(32 * ((rt + 1) * blocks / row_tiles)), a.rows)};
  if (a.offsets) {
    tile = find_tile<T::kRows>(a.offsets, a.experts, a.rows, rt, lane);
    if (tile.expert < 0) return;
  }

  // Its pairs of kb.
  const int pair0 = part * a.kp / split, kp = (part + 1) * a.kp / split - pair0;
  const int kbs = min((a.k >> 7) - 2 * pair0, 2 * kp);

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
    const int64_t unit = (int64_t)rb * a.kp + pair0;
    wb[i] = a.w + tile.expert * a.w_bytes + unit * (4 * T::kStepW);
    wsb[i] = a.ws + tile.expert * a.ws_bytes + unit * 256;
  }
  const int x_row = FX == MXG_MXFP4 ? a.k >> 1 : a.k;
  const int64_t base_row = a.gather ? 0 : tile.r0;
  const uint8_t* xb = a.x + base_row * x_row + (int64_t)pair0 * (T::kStages * T::kLine);
  const uint8_t* xsb = a.xs + base_row * (a.k >> 5) + (int64_t)pair0 * 8;
  const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int last = (kbs * 2 + T::kPer - 1) / T::kPer - 1;  // the last stage that x has

  // The tile with NX blocks of 32 rows of x for each wave: block t of wave column wx
  // is the tile's block t * WX + wx, so that a tile of few rows is shared evenly.
  auto run = [&](auto blocks) __attribute__((always_inline)) {
    constexpr int NX = decltype(blocks)::value;
    constexpr int kBlocks = WX * NX;
    constexpr int kCopyX = (kBlocks + T::kWaves - 1) / T::kWaves;
    constexpr int kWLoads = T::kWBlock / 1024;
    constexpr int kCopies = T::kCopyW + T::kXLoads * kCopyX;

    // Rows of x: a wave instruction takes 64 bytes of 16 rows, lane l the piece (l ^ l /
    // 8) % 4 of row l / 4, so that row r holds piece p at p ^ (r / 2) % 4 (or 128 of 8,
    // piece (l ^ l / 8) % 8 of row l / 8, at p ^ r % 8), and the lanes of an operand read
    // meet no bank twice. Rows past the end: the last one again. (Where the blocks do not
    // go round, two waves copy the same one.)
    constexpr int kPieces = T::kLine / 16;
    const uint32_t half = 64 * ((lane ^ (lane >> 3)) >> 2 & 1);
    uint32_t xo[kCopyX][T::kXLoads], xso[kCopyX];
    int xblock[kCopyX];
#pragma unroll
    for (int i = 0; i < kCopyX; ++i) {
      const int b = xblock[i] = (wave + i * T::kWaves) % kBlocks;
#pragma unroll
      for (int j = 0; j < T::kXLoads; ++j) {
        const int row =
            min(tile.r0 + 32 * b + (32 / T::kXLoads) * j + lane / kPieces, tile.r1 - 1);
        xo[i][j] = (uint32_t)(source_row(a, row) - base_row) * (uint32_t)x_row +
                   16 * ((lane ^ (lane >> 3)) & (kPieces - 1));
      }
      const int row = min(tile.r0 + 32 * b + r32, tile.r1 - 1);
      xso[i] = (uint32_t)(source_row(a, row) - base_row) * (uint32_t)(a.k >> 5) + 4 * g;
    }

    // Copy n of a stage: W's blocks, x's (two each), with a pair's first stage its
    // scales. Where K ends with a pair's first half, W is zero in the second, and x's
    // codes (by `half`, where a stage is a whole pair) and scales before it are taken
    // again.
    auto copy = [&](int n, int stage) __attribute__((always_inline)) {
      const uint32_t to = base + (uint32_t)stage % T::kRing * T::kSlot;
      const int pair = stage / T::kStages;
      const uint32_t sto = base + T::kScales + (pair & (T::kScaleRing - 1)) * T::kPair;
      if (n < T::kCopyW) {
        copy_kib<kWLoads>(to + (wave + n * T::kWaves) * T::kWBlock,
                          wb[n] + (int64_t)stage * T::kWBlock, 16 * lane);
      } else if (n < kCopies) {
        const int i = (n - T::kCopyW) / T::kXLoads, j = (n - T::kCopyW) % T::kXLoads;
        uint32_t from = xo[i][j];
        if (T::kPer == 4 && stage == last && kbs & 1) from -= half;
        copy_kib<1>(to + T::kX + xblock[i] * T::kXBlock + 1024 * j,
                    xb + (int64_t)min(stage, last) * T::kLine, from);
      } else if (n < kCopies + T::kCopyW) {
        const int i = n - kCopies;
        copy_words(sto + (wave + i * T::kWaves) * 256, wsb[i] + (int64_t)pair * 256, 4 * lane);
      } else {
        const int i = n - kCopies - T::kCopyW;
        copy_words(sto + (T::kNW + xblock[i]) * 256, xsb + (int64_t)pair * 8,
                   xso[i] - (2 * pair + 1 < kbs ? 0 : 4 * g));
      }
    };
    // Part `part` of `parts` of a stage's copies.
    auto copy_part = [&](int stage, bool scales, int part, int parts)
                         __attribute__((always_inline)) {
      const int all = kCopies + (scales ? T::kCopyW + kCopyX : 0);
#pragma unroll
      for (int n = part * all / parts; n < (part + 1) * all / parts; ++n) copy(n, stage);
    };

    // The first kAhead stages (with two steps a stage, the last one's second half comes
    // in the first step).
#pragma unroll
    for (int j = 0; j < T::kAhead; ++j)
      if (j < T::kStages * kp)
        copy_part(j, j % T::kStages == 0, 0, j == T::kAhead - 1 ? T::kPer : 1);

    v16f acc[RW][NX];
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int t = 0; t < NX; ++t) {
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][t][q] = 0.f;
        asm volatile("" : "+a"(acc[i][t]));  // here, under the loads' latency
      }
    // Operands of this and the next step; W's of the next one take the registers of
    // this one's where MFMAs are long enough (MXFP8: 64 cycles) to hide the reads after
    // the last use (two sets of both are more registers than there are).
    constexpr int kSetsW = FX == MXG_MXFP8 ? 1 : 2;
    Piece<FW> opw[kSetsW][RW];
    Piece<FX> opx[2][NX];
    uint32_t sw[RW], sx[NX];

    const uint32_t w_at = ww * RW * T::kWBlock + 16 * lane;
    const uint32_t x_at = T::kX + wx * T::kXBlock + T::kLine * r32 +
                          16 * (g ^ (T::kLine == 64 ? r32 >> 1 & 3 : r32 & 7));
    auto lds16 = [&](uint32_t at) __attribute__((always_inline)) {
      return *reinterpret_cast<const v4u*>(lds + at);
    };
    // The n-th operand of step S of a pair whose first stage is `first`: W's, then x's.
    auto fetch = [&](int n, auto step, int first) __attribute__((always_inline)) {
      constexpr int S = decltype(step)::value;
      Piece<FW>* const w = opw[S % kSetsW];
      Piece<FX>* const x = opx[S & 1];
      const uint32_t slot = (uint32_t)(first + S / T::kPer) % T::kRing * T::kSlot;
      if (n < RW) {
        const uint32_t p = slot + w_at + n * T::kWBlock + (S % T::kPer) * T::kStepW;
        w[n].lo = lds16(p);
        if constexpr (FW == MXG_MXFP8) w[n].hi = lds16(p + 1024);
      } else {
        const int t = n - RW;
        const uint32_t p = slot + t * WX * T::kXBlock;
        const uint32_t at = x_at ^ (T::kLine / T::kPer * (S % T::kPer));
        x[t].lo = lds16(p + at);
        if constexpr (FX == MXG_MXFP8) x[t].hi = lds16(p + (at ^ 32));
      }
    };
    // A pair's scales, byte S of a word that of step S.
    auto fetch_scales = [&](uint32_t (&w)[RW], uint32_t (&x)[NX], int pair)
                            __attribute__((always_inline)) {
      const uint8_t* p = lds + T::kScales + (pair & (T::kScaleRing - 1)) * T::kPair;
#pragma unroll
      for (int i = 0; i < RW; ++i)
        w[i] = *reinterpret_cast<const uint32_t*>(p + (ww * RW + i) * 256 + 4 * lane);
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        const uint32_t* q =
            reinterpret_cast<const uint32_t*>(p + (T::kNW + wx + t * WX) * 256 + 4 * r32);
        x[t] = __builtin_amdgcn_perm(q[32], q[0], g ? 0x07050301u : 0x06040200u);
      }
    };

    // One step of a pair: its products, between them the next step's operands and
    // copies. LEFT: the pairs there are after this one (2: or more). Before a stage's
    // last step its operands are in registers in every wave that has passed the barrier,
    // so its slot is free for another stage; there the next stage has to have landed,
    // younger loads may still fly.
    auto step = [&](auto number, auto left, int pair) __attribute__((always_inline)) {
      constexpr int S = decltype(number)::value, kLeft = decltype(left)::value;
      constexpr int kM = RW * NX, P = T::kPer;
      constexpr bool kEdge = S % P == P - 1;  // a stage's last step
      constexpr bool kNext = S < 3 || kLeft > 0;
      constexpr int J = S / P;                      // its stage of the pair
      const int first = pair * T::kStages;
      // Whether stage q, counted from this pair's first one, exists: q < kThere.
      constexpr int kThere = kLeft == T::kLefts ? 99 : (kLeft + 1) * T::kStages;
      uint32_t nw[RW], nx[NX];
      if constexpr (kEdge && kNext) {
        constexpr int kEnd = J + T::kAhead < kThere ? J + T::kAhead : kThere;
        wait_loads<T::loads(J + 2, kEnd, kCopyX)>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if constexpr (S == 3) fetch_scales(nw, nx, pair + 1);
      }
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        // Neighbouring products share an operand, which costs less energy.
        const int t = m / RW;
        const bool back = t % 2 == 1 && (kSetsW == 2 || t < NX - 1);
        const int i = back ? RW - 1 - m % RW : m % RW;
        acc[i][t] = product<FW, FX, S, S>(opw[S % kSetsW][i], sw[i], opx[S & 1][t], sx[t],
                                          acc[i][t]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kNext) {
          const int then = first + (S == 3 ? T::kStages : 0);
          if (kSetsW == 2) {
#pragma unroll
            for (int n = m * (RW + NX) / kM; n < (m + 1) * (RW + NX) / kM; ++n)
              fetch(n, Int<(S + 1) % 4>(), then);
          } else {
            // x's under the products before W's last uses (of one block: with the first).
            constexpr int kBefore = NX > 1 ? kM - RW : 1;
            if (m >= kM - RW) fetch(i, Int<(S + 1) % 4>(), then);
#pragma unroll
            for (int n = m * NX / kBefore; n < (m + 1) * NX / kBefore && n < NX; ++n)
              fetch(RW + n, Int<(S + 1) % 4>(), then);
          }
        }
        // Stage J + kAhead: with two steps a stage, half in its last one, half in the next.
        constexpr int kTo = kEdge ? J + T::kAhead : J + T::kAhead - 1;
        if constexpr (kTo < kThere)
          copy_part(first + kTo, kTo % T::kStages == 0, kEdge ? m : kM * (S % P + 1) + m, kM * P);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (S == 3 && kNext) {
#pragma unroll
        for (int i = 0; i < RW; ++i) sw[i] = nw[i];
#pragma unroll
        for (int t = 0; t < NX; ++t) sx[t] = nx[t];
      }
    };
    auto whole = [&](auto left, int pair) __attribute__((always_inline)) {
      step(Int<0>(), left, pair);
      step(Int<1>(), left, pair);
      step(Int<2>(), left, pair);
      step(Int<3>(), left, pair);
    };

    // The first stage is there; of the others as many instructions may be in flight as
    // were issued.
    if (T::kStages * kp >= T::kAhead)
      wait_loads<T::loads(1, T::kAhead - 1, kCopyX) + T::first_half(T::kAhead - 1, kCopyX)>();
    else
      wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch_scales(sw, sx, 0);
#pragma unroll
    for (int n = 0; n < RW + NX; ++n) fetch(n, Int<0>(), 0);
    int pair = 0;
    for (; pair + T::kLefts < kp; ++pair) whole(Int<T::kLefts>(), pair);
    if constexpr (T::kLefts > 3)
      if (pair + 3 < kp) whole(Int<3>(), pair++);
    if constexpr (T::kLefts > 2)
      if (pair + 2 < kp) whole(Int<2>(), pair++);
    if constexpr (T::kLefts > 1)
      if (pair + 1 < kp) whole(Int<1>(), pair++);
    whole(Int<0>(), pair);
    // The sums are read no sooner than 32 wait states behind the last product: a guard. The
    // compiler counts 19 behind an MXFP8 product of 64 cycles, which is that product's length;
    // a form of this kernel with a wave more read the last product's last sum without it, and
    // the cause is not shown. (Small tiles by two run two waves on a SIMD as well; they have
    // not shown it.)
#pragma unroll
    for (int t = 0; t < NX; ++t)
#pragma unroll
      for (int i = 0; i < RW; ++i)
        if (t + i == 0)
          asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc[i][t]));
        else
          asm volatile("" : "+a"(acc[i][t]));

    // ---- epilogue
    if (T::kSplits && split > 1) {  // sums as they lie, 1 KiB a store, for join_kernel
      float4* to = reinterpret_cast<float4*>(a.partial) +
                   ((int64_t)(number * split + part) * T::kWaves + wave) * (RW * RX * 256) + lane;
#pragma unroll
      for (int t = 0; t < NX; ++t)
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            to[(t * RW + i) * 256 + 64 * q] =
                float4{acc[i][t][4 * q], acc[i][t][4 * q + 1], acc[i][t][4 * q + 2],
                       acc[i][t][4 * q + 3]};
      return;
    }
    // 32 rows of the wave's columns meet in LDS and go out by whole lines.
    __syncthreads();  // (the ring is read out)
    uint8_t* const mine = lds + wave * 32 * T::kOutRow;
    auto emit = [&](auto gate) __attribute__((always_inline)) {
      constexpr bool kTwo = decltype(gate)::value;
      constexpr int kWidth = (kTwo ? 16 : 32) * RW;  // columns of the wave
      constexpr int kLanes = kWidth / 8;             // of 16 bytes, for a row
      const int col = ct * (kTwo ? 16 : 32) * T::kNW + ww * kWidth + 8 * (lane % kLanes);
      constexpr int kTimes = 32 * kLanes / 64;  // stores of a lane for 32 rows
      int to[NX][kTimes];                       // (one round trip for each)
#pragma unroll
      for (int t = 0; t < NX; ++t)
#pragma unroll
        for (int u = 0; u < kTimes; ++u) {
          const int row = tile.r0 + 32 * (t * WX + wx) + lane / kLanes + u * (64 / kLanes);
          to[t][u] = row < tile.r1 ? target_row(a, row) : -1;
        }
#pragma unroll
      for (int t = 0; t < NX; ++t) {
        auto lay = [&](const v16f& v, int block) __attribute__((always_inline)) {
#pragma unroll
          for (int q = 0; q < 4; q += 2)
            *reinterpret_cast<uint4*>(mine + r32 * T::kOutRow + 64 * block + 16 * (q + g)) =
                eight_columns(v, q);
        };
        if constexpr (kTwo) {
#pragma unroll
          for (int i = 0; i < RW; i += 2) lay(gated(acc[i][t], acc[i + 1][t]), i / 2);
        } else {
#pragma unroll
          for (int i = 0; i < RW; ++i) lay(acc[i][t], i);
        }
        __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
        v4u v[kTimes];
#pragma unroll
        for (int u = 0; u < kTimes; ++u)
          v[u] = *reinterpret_cast<const v4u*>(
              mine + (lane / kLanes + u * (64 / kLanes)) * T::kOutRow + 16 * (lane % kLanes));
#pragma unroll
        for (int u = 0; u < kTimes; ++u)
          if (to[t][u] >= 0 && col < a.out_n)
            __builtin_nontemporal_store(
                v[u], reinterpret_cast<v4u*>(a.out + (int64_t)to[t][u] * a.out_n + col));
        __builtin_amdgcn_wave_barrier();
      }
    };
    if (a.gated)
      emit(Int<1>());
    else
      emit(Int<0>());
  };
  const int n = (tile.r1 - tile.r0 + 32 * WX - 1) / (32 * WX);
  if constexpr (RX == 8) {
    if (n == 8) return run(Int<8>());
    if (n == 7) return run(Int<7>());
    if (n == 6) return run(Int<6>());
    if (n == 5) return run(Int<5>());
    if (n == 4) return run(Int<4>());
    if (n == 3) return run(Int<3>());
  }
  static_assert(RX == 2 || RX == 8, "");
  if (n == 2)
    run(Int<2>());
  else
    run(Int<1>());
}

// Adds up the parts of a split K in ascending order. A wave takes 16 columns of 32
// rows of x (gated: of gate and up): a quarter of a block pair, so that there are
// enough waves for the memory.
template <int RW, int RX, int WW, int WX, bool GATED>
__global__ void __launch_bounds__(64) join_kernel(RowsArgs a, int row_tiles, int col_tiles,
                                                  int split) {
  constexpr int kWaves = WW * WX, kNW = WW * RW;
  constexpr int kN = GATED ? 2 : 1;
  const int lane = threadIdx.x, r32 = lane & 31, g = lane >> 5;
  const int t = blockIdx.x % RX, wave = blockIdx.x / RX % kWaves;
  const int number = blockIdx.x / (RX * kWaves);
  const int half = blockIdx.y % 2, block = blockIdx.y / 2;
  const int ww = wave % WW, wx = wave / WW;
  int ct, rt;
  tile_at(number, row_tiles, col_tiles, &ct, &rt);
  const int64_t blocks = (a.rows + 31) / 32;
  const int row = (int)(32 * (rt * blocks / row_tiles)) + 32 * (t * WX + wx);
  if (row >= min((int)(32 * ((rt + 1) * blocks / row_tiles)), a.rows)) return;
  const float4* from = reinterpret_cast<const float4*>(a.partial) +
                       ((int64_t)number * split * kWaves + wave) * (RW * RX * 256) +
                       (t * RW + block * kN) * 256 + 128 * half + lane;
  float s[kN][8] = {};
  constexpr int B = 8;  // parts in flight
  for (int p0 = 0; p0 < split; p0 += B) {
    float4 v[B][kN][2];
#pragma unroll
    for (int p = 0; p < B; ++p)
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          v[p][i][q] = from[(int64_t)min(p0 + p, split - 1) * (kWaves * RW * RX * 256) + i * 256 +
                            64 * q];
#pragma unroll
    for (int p = 0; p < B; ++p) {
      if (p0 + p >= split) break;
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          s[i][4 * q] += v[p][i][q].x;
          s[i][4 * q + 1] += v[p][i][q].y;
          s[i][4 * q + 2] += v[p][i][q].z;
          s[i][4 * q + 3] += v[p][i][q].w;
        }
    }
  }
  float h[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) h[q] = GATED ? gated(s[0][q], s[kN - 1][q]) : s[0][q];
  const uint4 u = eight_columns(h);
  const int c = 32 * ((ct * kNW + ww * RW) / kN + block) + 16 * half + 8 * g;
  if (row + r32 < a.rows && c < a.out_n)
    *reinterpret_cast<uint4*>(a.out + (int64_t)(row + r32) * a.out_n + c) = u;
}

template <int FW, int FX, int RW, int RX, int WW, int WX, bool DEEP>
hipError_t launch(const RowsArgs& a, const RowsChoice& h, hipStream_t s) {
  using T = Tile<FW, FX, RW, RX, WW, WX, DEEP>;
  static_assert(T::kRows == 32 * T::kNW, "");
  const TileGrid g = tile_grid(h.row_tiles * h.col_tiles * h.split);
  hipLaunchKernelGGL((rows_tile_kernel<FW, FX, RW, RX, WW, WX, DEEP>), dim3(g.x, g.y),
                     dim3(T::kThreads), 0, s, a, (int)h.row_tiles, (int)h.col_tiles, h.split);
  return hipGetLastError();
}

// (of tiles of 128 by 128)
hipError_t launch_join(const RowsArgs& a, const RowsChoice& h, hipStream_t s) {
  const dim3 joins((unsigned)(h.row_tiles * h.col_tiles * 8), a.gated ? 2 : 4);
  if (a.gated)
    hipLaunchKernelGGL((join_kernel<2, 2, 2, 2, true>), joins, dim3(64), 0, s, a,
                       (int)h.row_tiles, (int)h.col_tiles, h.split);
  else
    hipLaunchKernelGGL((join_kernel<2, 2, 2, 2, false>), joins, dim3(64), 0, s, a,
                       (int)h.row_tiles, (int)h.col_tiles, h.split);
  return hipGetLastError();
}

template <int FW, int FX>
hipError_t by_size(const RowsArgs& a, const RowsChoice& h, hipStream_t s) {
  if (h.side == 256) return launch<FW, FX, 2, 8, 4, 1, false>(a, h, s);
  return h.row_tiles * h.col_tiles * h.split <= 256 ? launch<FW, FX, 2, 2, 2, 2, true>(a, h, s)
                                                    : launch<FW, FX, 2, 2, 2, 2, false>(a, h, s);
}

}  // namespace

hipError_t launch_rows_tile(const RowsArgs& a, int w_format, int x_format, const RowsChoice& h,
                            hipStream_t s) {
  hipError_t e;
  if (x_format == MXG_MXFP4)
    e = by_size<MXG_MXFP4, MXG_MXFP4>(a, h, s);
  else if (x_format == MXG_MXFP8)
    e = launch_rows_bf16(a, w_format, (int)h.row_tiles, (int)h.col_tiles, h.split, s);
  else if (w_format == MXG_MXFP4)
    e = by_size<MXG_MXFP4, MXG_MXFP8>(a, h, s);
  else
    e = by_size<MXG_MXFP8, MXG_MXFP8>(a, h, s);
  return e == hipSuccess && h.split > 1 ? launch_join(a, h, s) : e;
}

}  // namespace mxg
