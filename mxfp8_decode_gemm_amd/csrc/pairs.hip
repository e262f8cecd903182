// A router's (token, choice) pairs (gfx950): mxmoe_sort and mxmoe_combine of
// include/mxrows.h.

#include <hip/hip_runtime.h>

#include "mx_device.h"
#include "rows_internal.h"

namespace mxg {
namespace {

// ---- sort --------------------------------------------------------------------
//
// A counting sort that keeps the order of equal keys (the only atomics add whole
// numbers in LDS). Workgroups take contiguous chunks of the pairs, waves contiguous
// parts of a chunk. Bucket e < experts holds expert e's pairs, bucket `experts` those
// without one. A pair's place is the sum of what lies before its bucket, of its bucket
// in earlier workgroups, in earlier waves and in earlier pairs of its wave; the last
// comes from matching the 64 keys of a round bit by bit.
//
// One workgroup does it in one launch. More of them count first, in a launch of
// their own (a row of the workspace each), and each then sums the rows itself:
// with at most kMostGroups of them that costs less than a third launch. The second
// launch reads and matches its keys again, to count before the workspace's rows and to
// place behind them.
//
// Bound by latency: 64 pairs 3.1 us, 1024 of 256 experts 4.1, 2048 5.6, 4096 8.4; by more
// than one workgroup 4104 pairs 7.6 (no workspace up to there), 131072 10.8 (12.7 and 15.3
// by chunks of 2048 and 4096), 300000 15.6.

constexpr int kSortWaves = 16;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kBuckets = MXG_MOE_MAX_EXPERTS + 2;  // an even number
constexpr int kOne = 4096;    // most pairs of a single workgroup
constexpr int kChunk = 1024;  // pairs of each of several, or more:
constexpr int kMostGroups = 256;

struct SortArgs {
  const int32_t* ids;
  int32_t pairs, experts, chunk, groups, stride;  // stride: words of a workspace row
  uint32_t* counts;                               // [groups][stride]
  int32_t *order, *offsets;
};

// The lanes whose key equals this lane's; bits: of the largest key.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int i = 0; i < bits; ++i) {
    const bool one = key >> i & 1;
    const uint64_t b = __ballot(one);
    m &= one ? b : ~b;
  }
  return m;
}

// The bucket of pair p, or one past all of them for p >= end.
__device__ __forceinline__ int bucket_of(const SortArgs& a, int p, int end) {
  if (p >= end) return a.experts + 1;
  const int e = a.ids[p];
  return (unsigned)e < (unsigned)a.experts ? e : a.experts;
}

// Counts of a wave's pairs into its row of LDS.
__device__ __forceinline__ void count_part(const SortArgs& a, int p0, int p1, int bits, int lane,
                                           uint32_t* row) {
  for (int p = p0; p < p1; p += 64) {
    const int b = bucket_of(a, p + lane, p1);
    const uint64_t m = same_key(b, bits);
    if (b <= a.experts && __builtin_ctzll(m) == lane) row[b] += (uint32_t)__popcll(m);
    __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
  }
}

template <bool ONE>  // one workgroup: counts and places in this launch
__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(SortArgs a, int count_only) {
  __shared__ uint32_t part[kSortWaves][kBuckets];
  __shared__ uint32_t sums[kSortWaves];
  __shared__ uint32_t total[2][ONE ? 1 : kBuckets];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int used = a.experts + 1;
  const int bits = 32 - __builtin_clz(a.experts + 1);
  const int c0 = blockIdx.x * a.chunk, c1 = min(c0 + a.chunk, a.pairs);
  const int per = ((c1 - c0 + kSortThreads - 1) / kSortThreads) * 64;  // pairs of a wave
  const int p0 = min(c0 + wave * per, c1), p1 = min(p0 + per, c1);
  for (int i = lane; i < used; i += 64) part[wave][i] = 0;
  __builtin_amdgcn_wave_barrier();
  count_part(a, p0, p1, bits, lane, part[wave]);
  __syncthreads();

  if (!ONE && count_only) {
    for (int b = tid; b < a.stride; b += kSortThreads) {
      uint32_t n = 0;
      if (b < used)
        for (int w = 0; w < kSortWaves; ++w) n += part[w][b];
      a.counts[(int64_t)blockIdx.x * a.stride + b] = n;
    }
    return;
  }

  // Buckets 2 tid and 2 tid + 1: all their pairs, and those of earlier workgroups.
  uint32_t all[2] = {0, 0}, before[2] = {0, 0};
  if (ONE) {
    if (2 * tid < used) {
      for (int w = 0; w < kSortWaves; ++w) {
        all[0] += part[w][2 * tid];
        if (2 * tid + 1 < used) all[1] += part[w][2 * tid + 1];
      }
    }
  } else {
    // Teams of threads, one for each pair of buckets, take the workspace's rows in turn.
    const int half = a.stride / 2, teams = kSortThreads / half;
    const int team = tid / half, pair = tid - team * half;
    for (int b = tid; b < 2 * kBuckets; b += kSortThreads) total[b / kBuckets][b % kBuckets] = 0;
    __syncthreads();
    if (team < teams) {
      const uint2* row = reinterpret_cast<const uint2*>(a.counts) + pair;
      uint2 sum = {0, 0}, low = {0, 0};
#pragma unroll 8
      for (int k = team; k < a.groups; k += teams) {
        const uint2 n = row[(int64_t)k * half];
        const bool earlier = k < (int)blockIdx.x;
        sum.x += n.x;
        sum.y += n.y;
        low.x += earlier ? n.x : 0;
        low.y += earlier ? n.y : 0;
      }
      atomicAdd(&total[0][2 * pair], sum.x);
      atomicAdd(&total[0][2 * pair + 1], sum.y);
      atomicAdd(&total[1][2 * pair], low.x);
      atomicAdd(&total[1][2 * pair + 1], low.y);
    }
    __syncthreads();
    if (2 * tid < used) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        all[j] = total[0][2 * tid + j];
        before[j] = total[1][2 * tid + j];
      }
    }
  }
  const int mine = (int)(all[0] + all[1]);
  const int upto = wave_scan(mine);
  if (lane == 63) sums[wave] = (uint32_t)upto;
  __syncthreads();
  uint32_t at = (uint32_t)(upto - mine);
  for (int w = 0; w < wave; ++w) at += sums[w];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int b = 2 * tid + j;
    if (b >= used) break;
    if (blockIdx.x == 0) a.offsets[b] = (int32_t)at;
    uint32_t to = at + before[j];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t n = part[w][b];
      part[w][b] = to;
      to += n;
    }
    at += all[j];
  }
  __syncthreads();
  uint32_t* row = part[wave];
  for (int p = p0; p < p1; p += 64) {
    const int b = bucket_of(a, p + lane, p1);
    const uint64_t m = same_key(b, bits);
    const uint32_t first = b <= a.experts ? row[b] : 0;
    const uint32_t below = (uint32_t)__popcll(m & ((1ull << lane) - 1));
    __builtin_amdgcn_wave_barrier();
    if (b <= a.experts) {
      a.order[first + below] = p + lane;
      if (below == 0) row[b] = first + (uint32_t)__popcll(m);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

void sort_shape(int64_t pairs, int experts, int* chunk, int* groups, int* stride) {
  int64_t c = pairs <= kOne ? kOne : kChunk;
  if ((pairs + c - 1) / c > kMostGroups) c = (pairs + kMostGroups - 1) / kMostGroups;
  *chunk = (int)c;
  *groups = (int)((pairs + c - 1) / c);
  *stride = (experts + 2) / 2 * 2;
}

// ---- combine ------------------------------------------------------------------
//
// Bound by the read of y. One thread per 8 columns of a token; a token's ids and
// weights are the same for the whole workgroup (scalar loads), eight rows' loads in
// flight. Neighbouring workgroups take a token's columns: its rows lie together (4096
// tokens of 8 x 7168 81 us, 6.4 TB/s; 106 with neighbours along the tokens, level with
// 256 threads).

constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads)
    combine_pairs_kernel(const v4u* y, const int32_t* ids, const float* weights, int top_k,
                         int experts, int cols, int tokens, v4u* out) {
  const int c = blockIdx.x * kCombineThreads + threadIdx.x;
  if (c >= cols) return;
  for (int64_t t = blockIdx.y; t < tokens; t += gridDim.y) {
    float s[8] = {};
    constexpr int B = 8;
    const int64_t p0 = t * top_k;
    for (int j0 = 0; j0 < top_k; j0 += B) {
      // A pair without an expert takes the row of the first one that has one: every load
      // is issued, without a branch, and none of a row that is not asked for.
      int any = 0;
      float w[B];
      bool there[B];
#pragma unroll
      for (int j = B - 1; j >= 0; --j) {
        const int at = min(j0 + j, top_k - 1), e = ids[p0 + at];
        w[j] = weights[p0 + at];
        there[j] = j0 + j < top_k && (unsigned)e < (unsigned)experts;
        any = there[j] ? j + 1 : any;
      }
      if (any == 0) continue;
      v4u v[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        v[j] = __builtin_nontemporal_load(y + (p0 + j0 + (there[j] ? j : any - 1)) * cols + c);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = fmaf(w[j], __uint_as_float(u[i] << 16), s[2 * i]);
          const float b = fmaf(w[j], __uint_as_float(u[i] & 0xFFFF0000u), s[2 * i + 1]);
          s[2 * i] = there[j] ? a : s[2 * i];
          s[2 * i + 1] = there[j] ? b : s[2 * i + 1];
        }
      }
    }
    const v4u r = {bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]), bf16_pair(s[4], s[5]),
                   bf16_pair(s[6], s[7])};
    __builtin_nontemporal_store(r, out + t * cols + c);
  }
}

}  // namespace

size_t sort_workspace(int64_t pairs, int experts) {
  int chunk, groups, stride;
  sort_shape(pairs, experts, &chunk, &groups, &stride);
  if (groups == 1) return 0;
  return ((size_t)groups * stride * 4 + 15) / 16 * 16;
}

hipError_t launch_sort(const int32_t* ids, int pairs, int experts, void* workspace, int32_t* order,
                       int32_t* offsets, hipStream_t s) {
  SortArgs a;
  a.ids = ids;
  a.pairs = pairs;
  a.experts = experts;
  sort_shape(pairs, experts, &a.chunk, &a.groups, &a.stride);
  a.counts = static_cast<uint32_t*>(workspace);
  a.order = order;
  a.offsets = offsets;
  const dim3 grid((unsigned)a.groups), block(kSortThreads);
  if (a.groups == 1) {
    hipLaunchKernelGGL((sort_pairs_kernel<true>), grid, block, 0, s, a, 0);
  } else {
    hipLaunchKernelGGL((sort_pairs_kernel<false>), grid, block, 0, s, a, 1);
    hipLaunchKernelGGL((sort_pairs_kernel<false>), grid, block, 0, s, a, 0);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* y, const int32_t* ids, const float* weights, int tokens,
                          int top_k, int experts, int hidden, uint16_t* out, hipStream_t s) {
  const int cols = hidden / 8;
  const dim3 grid((unsigned)((cols + kCombineThreads - 1) / kCombineThreads),
                  (unsigned)(tokens < 65535 ? tokens : 65535));
  hipLaunchKernelGGL(combine_pairs_kernel, grid, dim3(kCombineThreads), 0, s,
                     reinterpret_cast<const v4u*>(y), ids, weights, top_k, experts, cols, tokens,
                     reinterpret_cast<v4u*>(out));
  return hipGetLastError();
}

}  // namespace mxg
