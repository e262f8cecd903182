// What the kernels that take tiles of many rows through LDS share (gfx950): copies
// without registers in between, counted waits, which tile a workgroup takes.
#pragma once

#include <type_traits>

#include "rows_device.h"

namespace mxg {
namespace {

// 1024 bytes from base + off (a lane's 16) to LDS at `to` (wave-uniform), and
// COUNT - 1 times the next 1024 to the next 1024. The compiler does not see these
// loads: their end is waited for with s_waitcnt vmcnt. (m0 is a reserved register: it
// cannot be named as clobbered, and the compiler writes it itself right before an
// instruction of its own that reads it, of which these kernels have none.)
template <int COUNT>
__device__ __forceinline__ void copy_kib(uint32_t to, const uint8_t* base, uint32_t off) {
  to = __builtin_amdgcn_readfirstlane(to);
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
                 "global_load_lds_dwordx4 %1, %2 offset:%3"
                 ::"s"(to), "v"(off), "s"(base), "n"(3 * 1024) : "memory");
}
// 256 bytes, 4 a lane.
__device__ __forceinline__ void copy_words(uint32_t to, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(to), "v"(off), "s"(base) : "memory");
}

// Tile `number` of a launch: eight row tiles side by side down the columns, so that
// neighbours share W and x.
__device__ __forceinline__ void tile_at(int number, int row_tiles, int col_tiles, int* ct,
                                        int* rt) {
  constexpr int kGroup = 8;
  const int group = row_tiles <= kGroup ? 0 : number / (kGroup * col_tiles);
  const int high = min(kGroup, row_tiles - group * kGroup);
  const int in = number - group * kGroup * col_tiles;
  *ct = high == kGroup ? in / kGroup : in / high;
  *rt = group * kGroup + (in - *ct * high);
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Workgroups go to the XCDs in turn: runs of 32 tiles stay on one, of fewer where
// there are not 256.
__device__ __forceinline__ int tile_of_workgroup() {
  const int run_of = min((int)gridDim.x / 8, kRun);
  const int bid = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  const int round = bid / (8 * kRun) * (8 * kRun);
  return round + (bid & 7) * run_of + ((bid - round) >> 3);
}

}  // namespace
}  // namespace mxg
