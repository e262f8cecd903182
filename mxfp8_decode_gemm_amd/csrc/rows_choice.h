// Which kernel a product of any number of rows runs on, by its sizes alone: a stream
// (rows_stream.hip), tiles of 128 or 256 (rows_tile.hip), or tiles in BF16
// (rows_bf16.hip). Plain C++: no HIP, host code may include it.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/mxrows.h"

namespace mxg {

// Units of the packed weight (rows_internal.h).
inline int unit_bytes(int format) { return format == MXG_MXFP4 ? 2048 : 4096; }
inline int64_t row_blocks(int64_t n) { return (n + 31) / 32; }
inline int64_t kb_pairs(int64_t k) { return (k + 255) / 256; }

struct RowsProblem {
  int64_t rows, nb, kp, w_bytes;  // of x; row blocks, pairs of kb and bytes of a weight
  int32_t experts, n;
  bool grouped, gated;
  bool w_fp4, x_fp4;
  bool bf16;  // MXFP8 rows that are not to be fast
};

inline RowsProblem rows_problem(int format, int x_format, int32_t experts, int32_t n, int32_t k,
                                bool gated, int64_t rows, bool grouped) {
  const int64_t nb = row_blocks(n), kp = kb_pairs(k);
  return {rows,    nb,    kp,    nb * kp * 2 * unit_bytes(format), experts, n,
          grouped, gated, format == MXG_MXFP4, x_format == MXG_MXFP4, x_format == MXG_MXFP8};
}

// What a launch is cut into: streams, or tiles of `side` rows of W and of x, K in `split`
// parts.
struct RowsChoice {
  int side;  // 0: streams
  int64_t row_tiles, col_tiles;
  int split;
  double us;  // (of one weight)
};

constexpr int kRun = 32;  // tiles side by side on one XCD

// The grid of a launch of so many tiles, a workgroup each: whole runs, in rows of 2^20 where
// there are more (a row's threads have to be countable in 32 bits).
struct TileGrid {
  unsigned x, y;
};
inline TileGrid tile_grid(int64_t tiles) {
  const int64_t unit = tiles < 8 * kRun ? 8 : 8 * kRun, most = 1 << 20;
  const int64_t grid = (tiles + unit - 1) / unit * unit;
  if (grid <= most) return {(unsigned)grid, 1};
  return {(unsigned)most, (unsigned)((grid + most - 1) / most)};
}

// Bytes of the sums of a divided K.
inline size_t choice_workspace(const RowsChoice& c) {
  return c.split > 1 ? (size_t)(c.row_tiles * c.col_tiles) * c.split * 4 * c.side * c.side : 0;
}

inline int64_t groups_of(const RowsProblem& a) { return a.experts < a.rows ? a.experts : a.rows; }
inline int64_t row_tiles(const RowsProblem& a, int side) {
  return a.grouped ? a.rows / side + groups_of(a) : (a.rows + side - 1) / side;
}

// The times that choose between them, in us, fitted to one MI355X's with W and x past the
// caches (k in pairs of kb; MXFP4 and MXFP8 x). Tiles of 128, 256 or fewer: 4096 x 2048 6.3
// and 9.4, 4096 x 4096 12 and 17, 4096 x 16384 33 and 50. Two on a CU: 1536 rows of 4096 x
// 4096 24 and 34, 1024 of 7168 x 8192 43 and 63.
inline double small_time(int64_t tiles, double kp, bool fp4) {
  if (tiles <= 256) return 3 + kp * (fp4 ? 0.5 : 0.75);
  return (double)((tiles + 511) / 512) * (4 + kp * (fp4 ? 1.17 : 1.95));
}
// Tiles of 256 with `h` blocks of 32 rows of x: 7168 x 8192 by 2 31 and 52, by 4 40 and 64,
// by 8 62 and 94; 2048 rows of 4096 x 4096 (by 4) 24 and 35.
inline double wide_time(int64_t tiles, double h, double kp, bool fp4) {
  const double pair = fp4 ? 0.55 + 0.14 * h : 1 + 0.23 * h;
  return (double)((tiles + 255) / 256) * (4 + 0.9 * h + kp * pair);
}
// What a divided K adds: a launch, the parts and their FP32 sums, written and read. Rows of
// 4096 x 16384 in MXFP4 with 1, 2 and 4 parts: 128 33, 23 and 18; 256 33, 24 and 23; 512 35
// and 30; 512 of 4096 x 4096 13 and 20. 32 of 2048 x 8192 in MXFP8 16 with 16 parts, 64 12
// with 8.
inline double join_time(int split, double rows, double n) {
  return 3 + 0.4 * split + split * rows * n * 8 / 3.5e6;
}

// Tiles of 128 in BF16 (rows_bf16.hip) with up to 64 rows of x and with up to 128: 2048 x
// 2048 13.6 and 18.3, 4096 x 4096 22.6 and 31, 1024 x 8192 41 and 56; 224 of 8192 59 (MXFP4)
// and 65. With 2, 4 and 8 parts of 64 rows 128 rows of 1024 x 8192 25.8, 17.3 and 14.9, of 4096
// x 4096 18.5 and 17.1 with 2 and 4; 203 of 4096 x 16384 40.6 with 4 by 128, 47 with 2 by 64.
inline double bf16_time(int64_t tiles, int64_t rows, double kp) {
  return (double)((tiles + 255) / 256) * (rows <= 64 ? 4.4 + 1.15 * kp : 5.5 + 1.58 * kp);
}
inline double bf16_join_time(int split, double rows, double n) {
  return 2 + 0.2 * split + split * rows * n * 8 / 3.5e6;
}

inline RowsChoice tile_choice(const RowsProblem& a) {
  RowsChoice big = {256, row_tiles(a, 256), (a.nb + 7) / 8, 1, 0};
  RowsChoice s = {128, row_tiles(a, 128), (a.nb + 3) / 4, 1, 0};
  if (a.grouped) {
    // Groups end in tiles that are half empty on average; only many rows a group, and
    // more tiles than CUs, make up for the larger tile's. By 128 and by 256, MXFP4: 64 experts
    // of 4096 x 7168 gated with 128 rows 306 and 301 us, 256 462 and 398, 512 771 and 640; 64 of
    // 2048 x 2048 with 128 rows 56 and 68, 256 85 and 79, 512 145 and 129; 8 of 4096 x 2048 gated
    // with 256 rows (192 tiles) 17 and 25, 512 (320) 30 and 28, of 4096 x 7168 54 and 68, 96 and
    // 77. 32 of 1024 x 4096 with 256 rows (192 tiles) lose by it, 50 and 42.
    const int64_t groups = groups_of(a), tiles = (a.rows / 256 + groups / 2) * big.col_tiles;
    return !a.bf16 && a.rows / groups >= 256 && tiles >= 256 ? big : s;
  }
  const bool fp4 = a.x_fp4;
  const int64_t blocks = (a.rows + 31) / 32;
  const double read = 2.5 + (double)a.w_bytes / 6.2e6;  // W, once
  // Tiles of 128 rows of x, and in BF16 of 64 too, with K whole and divided.
  s.us = INFINITY;
  const int64_t col_tiles = s.col_tiles, most = s.row_tiles;
  for (int64_t row_tiles : {most, a.bf16 ? (blocks + 1) / 2 : most}) {
    const int64_t tiles = row_tiles * col_tiles, rows = (blocks + row_tiles - 1) / row_tiles * 32;
    for (int split = 1; split <= 16; split *= 2) {
      if (split > 1 && (tiles * split > 256 || a.kp < 2 * split)) break;
      const double kp = (double)a.kp / split;
      const double join = split == 1 ? 0
                          : a.bf16   ? bf16_join_time(split, (double)a.rows, a.n)
                                     : join_time(split, (double)a.rows, a.n);
      const double t =
          fmax(a.bf16 ? bf16_time(tiles, rows, kp) : small_time(tiles, kp, fp4), read) + join;
      if (t < s.us) s = RowsChoice{128, row_tiles, col_tiles, split, t};
    }
  }
  if (a.bf16) return s;
  // Of large tiles as many down the rows as the last round of workgroups has room for:
  // lower ones.
  const int64_t rounds = (big.row_tiles * big.col_tiles + 255) / 256;
  const int64_t fit = rounds * 256 / big.col_tiles;
  if (fit > big.row_tiles) big.row_tiles = fit < blocks ? fit : blocks;
  const double h = (double)((blocks + big.row_tiles - 1) / big.row_tiles);
  big.us = wide_time(big.row_tiles * big.col_tiles, h, a.kp, fp4);
  return big.us < s.us ? big : s;
}

// Whether a call streams W for few rows or runs by tiles of many, by the measured times of
// both, in us.
// One weight: a round of 256 workgroups, each of 32 rows of W and 32 of x, streams 4096 x
// 2048 4.9 and 6.7 (MXFP4 and MXFP8), 4096 x 4096 7.6 and 10.9, 4096 x 16384 25 and 39; with
// 16 rows 3.4 and 4.7, 5.5 and 7.5, 15 and 27; with 8 at most 13 and 24. Either side of the
// border, streamed and by tiles: 64 rows of 4096 x 4096 in MXFP4 7.6 and 10.2, 96 13.1 and
// 12.4; 32 of 7168 x 8192 12.6 and 12.8, 64 23 and 13, in MXFP8 16 15.8 and 16.1, 32 20.7
// and 16.3; 128 of 2048 x 2048 4.3 and 7.5, 256 8.6 and 7.6.
// Experts, 64 of 4096 x k gated, by rows of each: k 512, 1 row 25 and 15; k 2048, 1 and 4
// rows 36 and 34, 53 and 49 (MXFP8 54 and 63, 80 and 93), 8 rows 61 and 52; k 4096, 8 and 16
// rows 100 and 107, 138 and 105.
//
// MXFP8 rows in BF16, W in MXFP4 and in MXFP8. One weight: 4096 x 2048 3.7 and 4.4 with 8
// rows, 4.3 and 4.9 with 16, 5.2 and 6.2 with 32, 4096 x 16384 16 and 19, 17 and 23, 26 and
// 36. Either side of the border, streamed and by tiles: 32 rows of 7168 x 8192 14 and 19
// (MXFP8 20 and 23), 64 27 and 20 (36 and 24); 128 of 1024 x 8192 14.5 and 14.9 (19.3 and
// 14.9), of 4096 x 4096 15.6 and 17.1 (20.4 and 17.2), 256 28.9 and 22.4 (39 and 22).
// Experts, 64 of 4096 x 2048 gated: 8 rows 69 and 113 (99 and 132), 16 105 and 117 (143 and
// 135), 32 128 and 129 (177 and 147); of 2048 x 2048 8 rows 42 and 57 (58 and 67), 16 63 and
// 57 (91 and 70); 8 of 2048 x 2048 with 16 rows 8.1 and 14 (11 and 15), with 32 16 and 15 (20
// and 15).
inline bool streams(const RowsProblem& a, double tiles_us) {
  if (a.grouped) {
    const int64_t groups = groups_of(a), mean = a.rows / groups;
    const int64_t columns = groups * (a.gated ? a.nb / 2 : a.nb);
    if (a.bf16) return mean <= (columns <= 1024 ? 16 : 8);
    return (mean <= 4 && a.kp >= 8) || (mean <= 8 && a.kp >= 16);
  }
  const int64_t chunks = (a.rows + 31) / 32;
  double pair;
  if (a.bf16)
    pair = a.rows <= 8    ? (a.w_fp4 ? 0.22 : 0.27)
           : a.rows <= 16 ? (a.w_fp4 ? 0.24 : 0.32)
                          : (a.w_fp4 ? 0.37 : 0.55);
  else
    pair = a.rows <= 8    ? (a.x_fp4 ? 0.18 : 0.35)
           : a.rows <= 16 ? (a.x_fp4 ? 0.22 : 0.39)
                          : (a.x_fp4 ? 0.36 : 0.57);
  const double rounds = (double)((a.nb * chunks + 255) / 256);
  const double us = rounds * ((a.bf16 ? 2 : 1.5) + (double)a.kp * pair) +
                    (a.bf16 ? 0.3 * (double)(chunks - 1) : 0);
  return tiles_us >= us;
}

inline RowsChoice rows_choice(const RowsProblem& a) {
  const RowsChoice c = tile_choice(a);
  return streams(a, c.us) ? RowsChoice{} : c;
}

}  // namespace mxg
