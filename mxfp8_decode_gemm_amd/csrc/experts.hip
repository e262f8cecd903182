// The chosen experts' gated products (gfx950): mxmoe_experts of
// include/mxdecode.h.
//
//   h[p]   = silu(Wg[e] x[t]) * (Wu[e] x[t])      pair p = (t, j), e = ids[p]
//   out[t] = sum_j weights[p] W2[e] h[p]
//
// What bounds it: a decode step's pairs touch few rows per expert, so the time
// is the read of the active experts' weights. Both products run as one
// weight-streaming kernel each, then one small kernel sums the pairs.
//
//   * The pairs are sorted by expert; each active expert's rows are cut into
//     chunks of NC column tiles of an MFMA. An item is (expert, 32 WN rows of W,
//     chunk); a workgroup takes a contiguous run of items, so the weights are
//     read once, in order, and no workgroup waits for another.
//   * The eight waves of a workgroup are WN along W's rows times WK along K.
//     Each streams its K blocks of the items, one item after the other, through
//     a ring of kRing register slots that runs on over the items' ends: W tiles
//     as mxgemm_pack_weight lays them (a wave instruction reads 1 KiB of
//     contiguous HBM), the rows' K blocks from x or h (in L2).
//   * At an item's end the waves' partial tiles meet in LDS and are summed in
//     ascending K order.
//   * W is converted with its scales to exact BF16 values. x is BF16. h goes
//     from the first product to the second as high and low BF16 parts (hi =
//     bf16(h), lo = bf16(h - hi)), which take columns c and c + 8 of a column
//     tile: the second product sees h to 17 bits at no extra W traffic, where
//     one BF16 rounding of h would add as much error as the result's own.
//   * Few pairs (narrow): every wave sorts them for itself, and the rows are
//     read as they lie in x and h, 16 lines per load. Many rows per expert
//     (WIDE): that gather costs more than the W stream (address lookups: 64 per
//     load instead of 16), so one kernel sorts the pairs and copies x into the
//     order of the MFMA's B operand, 1 KiB contiguous per load, and the first
//     product writes h in that order.

#include <hip/hip_runtime.h>

#include <cmath>

#include "mx_device.h"
#include "mxdecode_internal.h"

namespace mxg {

// The plans of both products in the workspace (WIDE).
struct WidePlan {
  int slots;
  int expert[MXG_MOE_MAX_PAIRS];
  int off[MXG_MOE_MAX_PAIRS + 1];
  int first[2][MXG_MOE_MAX_PAIRS + 1];  // chunks of the first, the second product
  int tile[2][MXG_MOE_MAX_PAIRS + 1];   // column tiles of 16, of 8 rows
  int order[MXG_MOE_MAX_PAIRS];
};

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kColStride = 36;  // floats per column of a partial tile: 32 rows, padded
// Ring slots. Two measured best: the loop's code stays short (instruction
// fetches cost more at the start than a deeper ring gains in the stream) and 67
// KB per CU in flight cover the latency. 4 slots: 8 tokens 7168x2048 8 of 64
// 198 + 105 us against 202 + 104, 1 token 39 + 24 against 40 + 22.5, 3 tokens
// 896x384 2 of 8 8.5 + 6.2 against 6.9 + 5.8.
constexpr int kRing = 2;
constexpr int kNarrowPairs = 64;

// The pairs sorted by expert. Slot s: expert[s], its pairs order[off[s] ..
// off[s + 1]), its chunks first[s] .. first[s + 1]; tile[s] its first column
// tile in the product's packed rows (WIDE).
template <int N>
struct Plan {
  int expert[N];
  int off[N + 1], first[N + 1], tile[N + 1];
  int order[N];
};

// The sum of v over this lane and the ones below.
__device__ __forceinline__ int wave_scan(int v) {
#define MXG_DPP_ADD(C, MASK) v += __builtin_amdgcn_update_dpp(0, v, C, MASK, 0xF, true)
  MXG_DPP_ADD(0x111, 0xF);  // rows of 16, then across them
  MXG_DPP_ADD(0x112, 0xF);
  MXG_DPP_ADD(0x114, 0xF);
  MXG_DPP_ADD(0x118, 0xF);
  MXG_DPP_ADD(0x142, 0xA);
  MXG_DPP_ADD(0x143, 0xC);
#undef MXG_DPP_ADD
  return v;
}
__device__ __forceinline__ int wave_prefix(int v) { return wave_scan(v) - v; }

// Up to 64 pairs: one per lane, without a barrier. Every wave computes the
// whole plan and writes the same words, so each may read it after its own
// writes. Experts come in the order of their first pair, an expert's pairs in
// ascending order. Returns the slots. RC: rows per chunk.
template <int RC>
__device__ __forceinline__ int make_plan(Plan<kNarrowPairs>& p, const int32_t* ids, int pairs,
                                         int experts, int lane) {
  int e = lane < pairs ? ids[lane] : -1;
  if ((unsigned)e >= (unsigned)experts) e = -1;
  int below = 0, all = 0, lead = 0;  // pairs of the same expert; the first one's lane
  for (int j = pairs - 1; j >= 0; --j) {
    const bool same = __builtin_amdgcn_readlane(e, j) == e;
    all += same ? 1 : 0;
    below += same && j < lane ? 1 : 0;
    lead = same ? j : lead;
  }
  const bool first = e >= 0 && lead == lane;
  const int ch = (all + RC - 1) / RC;
  const int s = wave_prefix(first ? 1 : 0);
  const int no = wave_prefix(first ? all : 0), co = wave_prefix(first ? ch : 0);
  if (first) {
    p.expert[s] = e;
    p.off[s] = no;
    p.first[s] = co;
  }
  const int at = __shfl(no, lead, 64) + below;
  if (e >= 0) p.order[at] = lane;
  const int slots = __builtin_amdgcn_readlane(s + (first ? 1 : 0), 63);
  if (lane == 63) {
    p.off[slots] = no + (first ? all : 0);
    p.first[slots] = co + (first ? ch : 0);
  }
  __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
  return slots;
}

// Piece q (16 bytes, 8 values) of lane group grp in a 128-wide K block: the
// order in which a lane's A operand holds K (mxgemm_pack_weight).
__device__ __forceinline__ int piece_k(int q, int grp) {
  return 64 * (q >> 1) + 16 * grp + 8 * (q & 1);
}

// Sorts the pairs and copies the rows of x into column tiles of 16:
// xp[tile][K block][q][grp][column] in 16-byte pieces. Every workgroup sorts
// for itself; the first one writes the plan out. 2^log0, 2^log1: rows per chunk.
// 2^share threads compare a pair with all others (in LDS, four at a time), with
// more than 512 pairs each thread does so for two; experts come in the order of
// their first pair, an expert's pairs in ascending order.
template <int kPer>
__global__ void __launch_bounds__(kThreads) sort_kernel(ExpertArgs a, int log0, int log1,
                                                        int share) {
  __shared__ __attribute__((aligned(16))) int sid[MXG_MOE_MAX_PAIRS];
  __shared__ int lead_off[MXG_MOE_MAX_PAIRS];   // of a first pair: its expert's place
  __shared__ int slot_of[MXG_MOE_MAX_PAIRS];    // of a column tile of 16
  __shared__ int totals[kPer][kWaves][3];
  __shared__ WidePlan p;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = a.tokens * a.top_k;
  const int padded = (pairs + 3) & ~3;
  const int part = tid & ((1 << share) - 1);
  int pair[kPer], e[kPer], below[kPer], all[kPer], lead[kPer], v[kPer][6];
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    pair[r] = r * kThreads + (tid >> share);
    e[r] = pair[r] < pairs ? a.ids[pair[r]] : -1;
    if ((unsigned)e[r] >= (unsigned)a.experts) e[r] = -1;
    if (part == 0 && pair[r] < padded) sid[pair[r]] = e[r];
    below[r] = all[r] = 0;
    lead[r] = MXG_MOE_MAX_PAIRS;
  }
  __syncthreads();
#pragma unroll 4
  for (int j = 4 * part; j < padded; j += 4 << share) {
    const int4 o = *reinterpret_cast<const int4*>(sid + j);
    const int ov[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool same = ov[q] == e[r];
        all[r] += same ? 1 : 0;
        below[r] += same && j + q < pair[r] ? 1 : 0;
        lead[r] = same ? min(lead[r], j + q) : lead[r];
      }
    }
  }
  for (int o = 1; o < 1 << share; o <<= 1) {  // (share > 0 only with one pair per thread)
    all[0] += __shfl_xor(all[0], o, 64);
    below[0] += __shfl_xor(below[0], o, 64);
    lead[0] = min(lead[0], __shfl_xor(lead[0], o, 64));
  }
  // Places of the experts: prefix sums over the first pairs, two sums in a word
  // (each at most 1024).
  int own[kPer][3];
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int c = e[r] >= 0 && below[r] == 0 && part == 0 ? all[r] : 0;
    own[r][0] = c | (c > 0 ? 1 : 0) << 16;
    own[r][1] = (c + (1 << log0) - 1) >> log0 | ((c + (1 << log1) - 1) >> log1) << 16;
    own[r][2] = (c + 15) >> 4 | ((c + 7) >> 3) << 16;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int to = wave_scan(own[r][k]);
      if (lane == 63) totals[r][wave][k] = to;
      v[r][2 * k] = to - own[r][k];  // for now both sums
    }
  }
  __syncthreads();
  int sum[3] = {};  // over all pairs
#pragma unroll
  for (int r = 0; r < kPer; ++r)
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (w == wave) v[r][2 * k] += sum[k];
        sum[k] += totals[r][w][k];
      }
  int end[6];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    end[2 * k] = sum[k] & 0xFFFF;
    end[2 * k + 1] = sum[k] >> 16;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      v[r][2 * k + 1] = v[r][2 * k] >> 16;
      v[r][2 * k] &= 0xFFFF;
    }
  }
  auto put = [&](const int (&u)[6]) __attribute__((always_inline)) {
    p.off[u[1]] = u[0];
    p.first[0][u[1]] = u[2];
    p.first[1][u[1]] = u[3];
    p.tile[0][u[1]] = u[4];
    p.tile[1][u[1]] = u[5];
  };
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    if (e[r] < 0 || below[r] != 0 || part != 0) continue;
    lead_off[pair[r]] = v[r][0];
    p.expert[v[r][1]] = e[r];
    put(v[r]);
    for (int t = 0; t < (all[r] + 15) >> 4; ++t) slot_of[v[r][4] + t] = v[r][1];
  }
  const int slots = end[1];
  if (tid == 0) put(end);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kPer; ++r)
    if (e[r] >= 0 && part == 0) p.order[lead_off[lead[r]] + below[r]] = pair[r];
  __syncthreads();
  if (blockIdx.x == 0) {
    WidePlan& g = *a.plan;
    if (tid == 0) g.slots = slots;
    for (int i = tid; i <= slots; i += kThreads) {
      if (i < slots) g.expert[i] = p.expert[i];
      g.off[i] = p.off[i];
      g.first[0][i] = p.first[0][i];
      g.first[1][i] = p.first[1][i];
      g.tile[0][i] = p.tile[0][i];
      g.tile[1][i] = p.tile[1][i];
    }
    for (int i = tid; i < end[0]; i += kThreads) g.order[i] = p.order[i];
  }
  // One wave per (tile, quarter of a K block): lane = (grp, column).
  const int K = a.hidden, pieces = K >> 5;  // 1 KiB pieces per tile
  const int col = lane & 15, grp = lane >> 4;
  const int units = end[4] * pieces;
  for (int u = blockIdx.x * kWaves + wave; u < units; u += gridDim.x * kWaves) {
    const int t = u / pieces, q = u - t * pieces;
    const int s = slot_of[t];
    const int pos = p.off[s] + 16 * (t - p.tile[0][s]) + col;
    if (pos >= p.off[s + 1]) continue;
    const int row = p.order[pos] / a.top_k;
    const int k = (q >> 2) * 128 + piece_k(q & 3, grp);
    a.xp[(size_t)u * 64 + lane] = *reinterpret_cast<const uint4*>(a.x + (size_t)row * K + k);
  }
}

// A position in the workgroup's run of items.
struct Walk {
  int slot, tile, chunk, chunks;

  template <typename P>
  __device__ __forceinline__ void enter(const P& p) {
    chunks = __builtin_amdgcn_readfirstlane(p.first[slot + 1] - p.first[slot]);
  }
  template <typename P>
  __device__ __forceinline__ void start(const P& p, int slots, int64_t item, int tiles) {
    int lo = 0, hi = slots;  // first[lo] * tiles <= item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      const int64_t f = (int64_t)__builtin_amdgcn_readfirstlane(p.first[mid]) * tiles;
      if (f <= item)
        lo = mid;
      else
        hi = mid;
    }
    slot = lo;
    enter(p);
    const int r = (int)(item - (int64_t)__builtin_amdgcn_readfirstlane(p.first[lo]) * tiles);
    tile = r / chunks;
    chunk = r - tile * chunks;
  }
  // The next item; true where its rows differ from the last one's.
  template <typename P>
  __device__ __forceinline__ bool next(const P& p, int tiles) {
    if (++chunk < chunks) return true;
    chunk = 0;
    if (++tile < tiles) return chunks > 1;
    tile = 0;
    ++slot;
    enter(p);
    return true;
  }
};

// UP: h from x and W13: wave wn takes the row blocks b = tile * WN + wn of the
// gate and inter / 16 + b of up. Otherwise y from h and W2, row blocks 2 b and
// 2 b + 1. NC: column tiles (16 rows, or 8 in two parts) per chunk.
template <bool UP, bool WIDE, int NC, int WK>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
experts_kernel(ExpertArgs a) {
  constexpr int WN = kWaves / WK;
  constexpr int RT = UP ? 16 : 8;  // rows per column tile
  constexpr int RC = RT * NC;      // rows per chunk
  constexpr int NBUF = NC > 2 ? 1 : 2;
  using PlanT = Plan<WIDE ? MXG_MOE_MAX_PAIRS : kNarrowPairs>;
  __shared__ PlanT plan;
  __shared__ __attribute__((aligned(16))) float red[NBUF][kWaves][NC * 16 * kColStride];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wk = wave / WN;
  const int r16 = lane & 15;
  const int grp = lane >> 4;
  const int pairs = a.tokens * a.top_k;
  const int K = UP ? a.hidden : a.inter;
  const int KBT = K >> 7;
  const int blocks = UP ? a.inter >> 4 : a.hidden >> 5;  // of 32 rows
  const int tiles = blocks / WN;

  int slots;
  if constexpr (WIDE) {
    const WidePlan& g = *a.plan;
    slots = __builtin_amdgcn_readfirstlane(g.slots);
    for (int i = tid; i <= slots; i += kThreads) {
      if (i < slots) plan.expert[i] = g.expert[i];
      plan.off[i] = g.off[i];
      plan.first[i] = g.first[UP ? 0 : 1][i];
      plan.tile[i] = g.tile[1][i];  // where h lies
      if (UP && i < slots) plan.order[i] = g.tile[0][i];  // where its x lies
    }
    if constexpr (!UP)
      for (int i = tid; i < pairs; i += kThreads) plan.order[i] = g.order[i];
    __syncthreads();
  } else {
    slots = make_plan<RC>(plan, a.ids, pairs, a.experts, lane);
  }
  const int64_t items = (int64_t)__builtin_amdgcn_readfirstlane(plan.first[slots]) * tiles;
  const int64_t item0 = items * blockIdx.x / gridDim.x;
  const int64_t item1 = items * (blockIdx.x + 1) / gridDim.x;
  if (item0 >= item1) return;

  const int kb0 = (wk * KBT) / WK;
  const int nbw = ((wk + 1) * KBT) / WK - kb0;
  const int nst = (nbw + kRing - 1) / kRing * kRing;  // ring steps per item
  const uint8_t* w = UP ? a.w13 : a.w2;
  const uint8_t* ws = UP ? a.w13s : a.w2s;
  const size_t wbytes = UP ? a.w13_bytes : a.w2_bytes;
  const size_t wsbytes = UP ? a.w13s_bytes : a.w2s_bytes;

  // ---- load side ---------------------------------------------------------
  Walk lw;
  lw.start(plan, slots, item0, tiles);
  int64_t litem = item0;
  int lkb = 0;
  bool live = true;
  __amdgpu_buffer_rsrc_t wrs[2], srs[2], brs;
  if constexpr (!WIDE)
    brs = __builtin_amdgcn_make_buffer_rsrc((void*)(UP ? a.x : a.h), (short)0,
                                            UP ? a.tokens * K * 2 : 2 * pairs * K * 2,
                                            kBufferWord3);
  int bvo[NC];  // this lane's columns of the chunk: byte offsets of their values
  auto set_rows = [&]() __attribute__((always_inline)) {
    const int b = plan.off[lw.slot] + lw.chunk * RC;
    const int n = plan.off[lw.slot + 1] - b;
    if constexpr (WIDE) {
      const int t0 = __builtin_amdgcn_readfirstlane(
          (UP ? plan.order[lw.slot] : plan.tile[lw.slot]) + lw.chunk * NC);
      brs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)((UP ? reinterpret_cast<const uint8_t*>(a.xp)
                      : reinterpret_cast<const uint8_t*>(a.h)) +
                  (size_t)t0 * K * 32),
          (short)0, NC * K * 32, kBufferWord3);
    }
#pragma unroll
    for (int t = 0; t < NC; ++t) {
      const int c = RT * t + (UP ? r16 : (r16 & 7));
      bvo[t] = kPastBuffer;
      if (c < n) {
        if constexpr (WIDE) {
          bvo[t] = t * K * 32 + 16 * lane;
        } else {
          const int p = plan.order[b + c];
          bvo[t] = (UP ? p / a.top_k : (r16 >> 3) * pairs + p) * K * 2 + 32 * grp;
        }
      }
    }
  };
  auto set_tile = [&]() __attribute__((always_inline)) {
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[lw.slot]);
    const int blk = lw.tile * WN + wn;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rb = UP ? blk + i * blocks : 2 * blk + i;
      const size_t t0 = (size_t)rb * KBT + kb0;
      wrs[i] = __builtin_amdgcn_make_buffer_rsrc((void*)(w + e * wbytes + t0 * 2048), (short)0,
                                                 nbw * 2048, kBufferWord3);
      srs[i] = __builtin_amdgcn_make_buffer_rsrc((void*)(ws + e * wsbytes + t0 * 64), (short)0,
                                                 nbw * 64, kBufferWord3);
    }
  };
  set_rows();
  set_tile();
  v4u wlo[kRing][2], whi[kRing][2], bx[kRing][NC][4];
  uint32_t wsc[kRing][2];
  // One K block into ring slot d; past the wave's K blocks and past the run's
  // end the offsets lie past the buffers (zeros, no memory access), so every
  // step issues the same loads.
  auto load = [&](int d) __attribute__((always_inline)) {
    const bool real = live && lkb < nbw;
    const int vo = real ? 16 * lane : kPastBuffer;
    const int so = real ? 4 * r16 : kPastBuffer;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wlo[d][i] = __builtin_amdgcn_raw_buffer_load_b128(wrs[i], vo, lkb * 2048, kLoadNontemporal);
      whi[d][i] =
          __builtin_amdgcn_raw_buffer_load_b128(wrs[i], vo + 1024, lkb * 2048, kLoadNontemporal);
      wsc[d][i] = __builtin_amdgcn_raw_buffer_load_b32(srs[i], so, lkb * 64, 0);
    }
    // Pieces q of the K block: 16 bytes of a row at piece_k, or 1 KiB apart.
    const int bk = (kb0 + lkb) * (WIDE ? 4096 : 256);
#pragma unroll
    for (int t = 0; t < NC; ++t) {
      const int bo = real ? bvo[t] : kPastBuffer;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bx[d][t][q] = __builtin_amdgcn_raw_buffer_load_b128(
            brs, bo + (WIDE ? 1024 * q : 128 * (q >> 1) + 16 * (q & 1)), bk, 0);
    }
    if (live && ++lkb == nst) {
      lkb = 0;
      if (++litem < item1) {
        if (lw.next(plan, tiles)) set_rows();
        set_tile();
      } else {
        live = false;
      }
    }
  };

  // ---- consume side --------------------------------------------------------
  Walk cw;
  cw.start(plan, slots, item0, tiles);
  int64_t citem = item0;
  int buf = 0;
  v4f acc[NC][2];
#pragma unroll
  for (int t = 0; t < NC; ++t) acc[t][0] = acc[t][1] = v4f{0.f, 0.f, 0.f, 0.f};
  const int sb0 = grp >> 1;  // 32-block of this lane's first 16 K (its second is sb0 + 2)
  auto consume = [&](int d) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f0 = e8m0_to_f32((wsc[d][i] >> (8 * sb0)) & 0xFFu);
      const float f1 = e8m0_to_f32((wsc[d][i] >> (8 * (sb0 + 2))) & 0xFFu);
      const v8bf av[4] = {fp8x8_to_bf16(wlo[d][i].x, wlo[d][i].y, f0),
                          fp8x8_to_bf16(wlo[d][i].z, wlo[d][i].w, f0),
                          fp8x8_to_bf16(whi[d][i].x, whi[d][i].y, f1),
                          fp8x8_to_bf16(whi[d][i].z, whi[d][i].w, f1)};
#pragma unroll
      for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              av[q], __builtin_bit_cast(v8bf, bx[d][t][q]), acc[t][i], 0, 0, 0);
    }
  };
  // The item's partial tiles -> LDS (with two buffers a wave writes one again
  // only after the barrier of the item between, which every wave reaches after
  // reading it), their sum in ascending K order, the epilogue.
  auto finish = [&]() __attribute__((always_inline)) {
    const int c0 = cw.chunk * RC;  // the chunk's first row among the expert's
    const int b = __builtin_amdgcn_readfirstlane(plan.off[cw.slot]) + c0;
    int n = __builtin_amdgcn_readfirstlane(plan.off[cw.slot + 1]) - b;
    n = n < RC ? n : RC;
    if constexpr (NBUF == 1) __syncthreads();
#pragma unroll
    for (int t = 0; t < NC; ++t) {
      if (RT * t + (UP ? r16 : (r16 & 7)) < n) {
        float* q = &red[buf][wave][(16 * t + r16) * kColStride + 4 * grp];
        *reinterpret_cast<v4f*>(q) = acc[t][0];
        *reinterpret_cast<v4f*>(q + 16) = acc[t][1];
      }
      acc[t][0] = acc[t][1] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();
    if constexpr (UP) {
      const int row = tid & 15;
      for (int i = tid >> 4; i < n * WN; i += kThreads / 16) {
        const int col = i / WN, g = i % WN;
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < WK; ++v) {
          gate += red[buf][v * WN + g][col * kColStride + row];
          up += red[buf][v * WN + g][col * kColStride + 16 + row];
        }
        const float h = gate / (1.f + expf(-gate)) * up;
        const __bf16 hi = (__bf16)h;
        // A high part beyond BF16's range has no remainder.
        const __bf16 lo = fabsf((float)hi) < INFINITY ? (__bf16)(h - (float)hi) : (__bf16)0.f;
        const int k = 16 * (cw.tile * WN + g) + row;
        size_t at, to_lo;
        if constexpr (WIDE) {
          const int pos = c0 + col, kk = k & 127;
          at = (size_t)(plan.tile[cw.slot] + (pos >> 3)) * a.inter * 16 + (k >> 7) * 2048 +
               (2 * (kk >> 6) + ((kk >> 3) & 1)) * 512 + ((kk >> 4) & 3) * 128 + (pos & 7) * 8 +
               (kk & 7);
          to_lo = 64;
        } else {
          at = (size_t)plan.order[b + col] * a.inter + k;
          to_lo = (size_t)pairs * a.inter;
        }
        a.h[at] = __builtin_bit_cast(uint16_t, hi);
        a.h[at + to_lo] = __builtin_bit_cast(uint16_t, lo);
      }
    } else {
      const int row = tid & 31;
      for (int i = tid >> 5; i < n * WN; i += kThreads / 32) {
        const int col = i / WN, g = i % WN;
        const int c = (col >> 3) * 16 + (col & 7);  // its high part; the low one 8 on
        float y = 0.f;
#pragma unroll
        for (int v = 0; v < WK; ++v) {
          const float* q = red[buf][v * WN + g];
          y += q[c * kColStride + row] + q[(c + 8) * kColStride + row];
        }
        a.y[(size_t)plan.order[b + col] * a.hidden + 32 * (cw.tile * WN + g) + row] = y;
      }
    }
    if constexpr (NBUF > 1) buf ^= 1;
    if (++citem < item1) cw.next(plan, tiles);
  };

  // An item takes a whole number of turns of the ring (a K slice that does not
  // fill the last one steps over zeros), so that the epilogue stands once in
  // the code.
  if (nst > 0) {
#pragma unroll
    for (int d = 0; d < kRing; ++d) load(d);
  }
  while (citem < item1) {
    for (int s0 = 0; s0 < nst; s0 += kRing) {
#pragma unroll
      for (int d = 0; d < kRing; ++d) {
        consume(d);
        load(d);
      }
    }
    finish();
  }
}

// out[t] = sum_j weights[t, j] y[t, j], one thread per 4 columns; eight pairs'
// loads in flight.
__global__ void combine_kernel(ExpertArgs a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int cols = a.hidden >> 2;
  if (i >= (int64_t)a.tokens * cols) return;
  const int t = (int)(i / cols);
  const int c = (int)(i - (int64_t)t * cols);
  constexpr int B = 8;
  float s[4] = {};
  for (int j0 = 0; j0 < a.top_k; j0 += B) {
    int e[B];
    float w[B];
    float4 y[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int p = t * a.top_k + (j0 + j < a.top_k ? j0 + j : j0);
      e[j] = a.ids[p];
      w[j] = a.weights[p];
      y[j] = *reinterpret_cast<const float4*>(a.y + (size_t)p * a.hidden + 4 * c);
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      // (y of a pair without an expert was not written.)
      if (j0 + j >= a.top_k || (unsigned)e[j] >= (unsigned)a.experts) continue;
      s[0] = fmaf(w[j], y[j].x, s[0]);
      s[1] = fmaf(w[j], y[j].y, s[1]);
      s[2] = fmaf(w[j], y[j].z, s[2]);
      s[3] = fmaf(w[j], y[j].w, s[3]);
    }
  }
  const uint2 v = {bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
  *reinterpret_cast<uint2*>(a.out + (size_t)t * a.hidden + 4 * c) = v;
}

template <bool UP, bool WIDE, int NC>
void launch_product(const ExpertArgs& a, int cus, hipStream_t s) {
  // Fewer than two K blocks per wave leave ring slots empty: half the waves
  // along K, twice the rows.
  const bool half = (UP ? a.hidden : a.inter) < 2 * kWaves * 128;
  // One workgroup per CU (two: the same), never more than there can be items.
  const int64_t tiles = (UP ? a.inter >> 4 : a.hidden >> 5) / (half ? 2 : 1);
  const int64_t most = (int64_t)a.tokens * a.top_k * tiles;
  const dim3 grid((unsigned)(most < cus ? most : cus)), block(kThreads);
  if (half)
    hipLaunchKernelGGL((experts_kernel<UP, WIDE, NC, 4>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((experts_kernel<UP, WIDE, NC, 8>), grid, block, 0, s, a);
}

// Column tiles of 16 and of 8 rows there can be.
size_t most_tiles(int64_t pairs, int64_t experts, int64_t rows) {
  const int64_t full = pairs / rows + (experts < pairs ? experts : pairs);
  return (size_t)(full < pairs ? full : pairs);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// The workspace: the plan, x in column tiles, h (two BF16 parts; 32 bytes per K
// of a column tile, at least 4 per pair), y (FP32).
size_t experts_workspace(ExpertArgs* a, void* base) {
  const int64_t pairs = (int64_t)a->tokens * a->top_k;
  const size_t plan = round256(sizeof(WidePlan));
  const size_t xp = most_tiles(pairs, a->experts, 16) * a->hidden * 32;
  const size_t t8 = most_tiles(pairs, a->experts, 8);
  const size_t h = round256(t8 * a->inter * 32);
  const size_t y = (size_t)pairs * a->hidden * 4;
  uint8_t* p = static_cast<uint8_t*>(base);
  a->plan = reinterpret_cast<WidePlan*>(p);
  a->xp = reinterpret_cast<uint4*>(p + plan);
  a->h = reinterpret_cast<uint16_t*>(p + plan + xp);
  a->y = reinterpret_cast<float*>(p + plan + xp + h);
  return plan + xp + h + y;
}

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess)
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  const int64_t pairs = (int64_t)a.tokens * a.top_k;
  // Rows per expert to expect: W is read again (from the caches) for every
  // chunk of them.
  const double mean = (double)pairs / (a.experts < pairs ? a.experts : pairs);
  double rows = mean + 2.0 * std::sqrt(mean);
  if (rows > a.tokens) rows = a.tokens;
  if (pairs <= kNarrowPairs && rows <= 8) {
    launch_product<true, false, 1>(a, cus, s);
    launch_product<false, false, 1>(a, cus, s);
  } else {
    const int nc0 = rows <= 16 ? 1 : 2, nc1 = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const size_t units = most_tiles(pairs, a.experts, 16) * (a.hidden >> 5);
    const size_t groups = (units + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(groups < 256 ? groups : 256)), block(kThreads);
    const int log0 = nc0 == 1 ? 4 : 5, log1 = nc1 == 1 ? 3 : nc1 == 2 ? 4 : 5;
    int share = 0;
    while (share < 4 && pairs << (share + 1) <= kThreads) ++share;
    if (pairs <= kThreads)
      hipLaunchKernelGGL((sort_kernel<1>), grid, block, 0, s, a, log0, log1, share);
    else
      hipLaunchKernelGGL((sort_kernel<2>), grid, block, 0, s, a, log0, log1, 0);
    if (nc0 == 1)
      launch_product<true, true, 1>(a, cus, s);
    else
      launch_product<true, true, 2>(a, cus, s);
    if (nc1 == 1)
      launch_product<false, true, 1>(a, cus, s);
    else if (nc1 == 2)
      launch_product<false, true, 2>(a, cus, s);
    else
      launch_product<false, true, 4>(a, cus, s);
  }
  const int64_t work = (int64_t)a.tokens * (a.hidden >> 2);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((work + 127) / 128)), dim3(128), 0, s, a);
  return hipGetLastError();
}

}  // namespace mxg
