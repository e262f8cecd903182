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
//   * Every workgroup first sorts the pairs by expert (in LDS): the active
//     experts in ascending order, each with its rows in chunks that fit the 16
//     columns of an MFMA. An item is (expert, two 16-row blocks of W, chunk);
//     a workgroup takes a contiguous run of items, so the weights are read
//     once, in order, and no workgroup waits for another.
//   * The eight waves of a workgroup split K. Each streams its K blocks of the
//     items, one after the other, through a ring of D registers slots that
//     runs on over the items' ends: W tiles as mxgemm_pack_weight lays them
//     (a wave instruction reads 1 KiB of contiguous HBM), the rows' K blocks
//     from x or h (small, in L2).
//   * At an item's end the waves' partial tiles meet in LDS and are summed in
//     ascending K order.
//   * W is converted with its scales to exact BF16 values. x is BF16. h goes
//     from the first product to the second as high and low BF16 parts (hi =
//     bf16(h), lo = bf16(h - hi)), which take columns c and c + 8 of the MFMA:
//     the second product sees h to 17 bits at no extra W traffic or MFMA, where
//     one BF16 rounding of h would add as much error as the result's own.

#include <hip/hip_runtime.h>

#include "mx_device.h"
#include "mxdecode_internal.h"

namespace mxg {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kColStride = 36;  // floats per column of a partial tile: 32 rows, padded

// The pairs sorted by expert. slot s: expert[s], its pairs order[off[s] ..
// off[s + 1]), its chunks first[s] .. first[s + 1].
struct Plan {
  int cnt[MXG_MOE_MAX_EXPERTS];
  int at[MXG_MOE_MAX_EXPERTS];
  int expert[MXG_MOE_MAX_PAIRS];
  int off[MXG_MOE_MAX_PAIRS + 1];
  int first[MXG_MOE_MAX_PAIRS + 1];
  int order[MXG_MOE_MAX_PAIRS];
  int slots;
};

__device__ __forceinline__ int wave_prefix(int v, int lane) {  // exclusive
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  return x - v;
}

// RC rows per chunk. The pairs of one expert stay in ascending order, so that
// every workgroup cuts them into the same chunks.
template <int RC>
__device__ void make_plan(Plan& p, const int32_t* ids, int pairs, int experts, int tid) {
  for (int e = tid; e < experts; e += kThreads) p.cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)experts) atomicAdd(&p.cnt[e], 1);
  }
  __syncthreads();
  if (tid < 64) {
    const int epl = (experts + 63) >> 6;
    const int lo = tid * epl, hi = min(lo + epl, experts);
    int n = 0, act = 0, ch = 0;
    for (int e = lo; e < hi; ++e) {
      const int c = p.cnt[e];
      n += c;
      act += c > 0 ? 1 : 0;
      ch += (c + RC - 1) / RC;
    }
    int no = wave_prefix(n, tid), s = wave_prefix(act, tid), co = wave_prefix(ch, tid);
    for (int e = lo; e < hi; ++e) {
      const int c = p.cnt[e];
      if (c == 0) continue;
      p.at[e] = no;
      p.expert[s] = e;
      p.off[s] = no;
      p.first[s] = co;
      no += c;
      co += (c + RC - 1) / RC;
      ++s;
    }
    if (tid == 63) {
      p.slots = s;
      p.off[s] = no;
      p.first[s] = co;
    }
  }
  __syncthreads();
  // 64 pairs at a time: a pair's place is its expert's next free one plus the
  // lower lanes of the same expert; the last of them moves the free place on.
  if (tid < 64) {
    for (int i0 = 0; i0 < pairs; i0 += 64) {
      const int i = i0 + tid;
      int e = i < pairs ? ids[i] : -1;
      if ((unsigned)e >= (unsigned)experts) e = -1;
      const int here = pairs - i0 < 64 ? pairs - i0 : 64;
      int below = 0, all = 0;
      for (int j = 0; j < here; ++j) {
        const int same = __builtin_amdgcn_readlane(e, j) == e ? 1 : 0;
        all += same;
        below += j < tid ? same : 0;
      }
      if (e >= 0) {
        const int at = p.at[e];
        p.order[at + below] = i;
        if (below == all - 1) p.at[e] = at + all;
      }
    }
  }
  __syncthreads();
}

// A position in the workgroup's run of items.
struct Walk {
  int slot, tile, chunk, chunks;

  __device__ __forceinline__ void enter(const Plan& p) {
    chunks = __builtin_amdgcn_readfirstlane(p.first[slot + 1] - p.first[slot]);
  }
  __device__ __forceinline__ void start(const Plan& p, int64_t item, int tiles) {
    int lo = 0, hi = __builtin_amdgcn_readfirstlane(p.slots);  // first[lo] * tiles <= item
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
  __device__ __forceinline__ bool next(const Plan& p, int tiles) {
    if (++chunk < chunks) return true;
    chunk = 0;
    if (++tile < tiles) return chunks > 1;
    tile = 0;
    ++slot;
    enter(p);
    return true;
  }
};

// UP: h from x and W13 (row blocks tile and inter / 16 + tile: gate and up).
// Otherwise: y from h and W2 (row blocks 2 tile and 2 tile + 1).
template <bool UP, int D>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2)))
experts_kernel(ExpertArgs a) {
  constexpr int RC = UP ? 16 : 8;  // rows per chunk
  __shared__ Plan plan;
  __shared__ __attribute__((aligned(16))) float red[2][kWaves][16 * kColStride];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15;
  const int grp = lane >> 4;
  const int pairs = a.tokens * a.top_k;
  const int K = UP ? a.hidden : a.inter;
  const int KBT = K >> 7;
  const int tiles = UP ? a.inter >> 4 : a.hidden >> 5;

  make_plan<RC>(plan, a.ids, pairs, a.experts, tid);
  const int slots = __builtin_amdgcn_readfirstlane(plan.slots);
  const int64_t items = (int64_t)__builtin_amdgcn_readfirstlane(plan.first[slots]) * tiles;
  const int64_t item0 = items * blockIdx.x / gridDim.x;
  const int64_t item1 = items * (blockIdx.x + 1) / gridDim.x;
  if (item0 >= item1) return;

  const int kb0 = (wave * KBT) / kWaves;
  const int nbw = ((wave + 1) * KBT) / kWaves - kb0;
  const uint8_t* w = UP ? a.w13 : a.w2;
  const uint8_t* ws = UP ? a.w13s : a.w2s;
  const size_t wbytes = UP ? a.w13_bytes : a.w2_bytes;
  const size_t wsbytes = UP ? a.w13s_bytes : a.w2s_bytes;
  const __amdgpu_buffer_rsrc_t brs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(UP ? a.x : a.h), (short)0, UP ? a.tokens * K * 2 : 2 * pairs * K * 2, kBufferWord3);

  // ---- load side ---------------------------------------------------------
  Walk lw;
  lw.start(plan, item0, tiles);
  int64_t litem = item0;
  int lkb = 0;
  bool live = nbw > 0;
  __amdgpu_buffer_rsrc_t wrs[2], srs[2];
  int bvo = kPastBuffer;  // this lane's column of the chunk: byte offset of its row
  auto set_rows = [&]() __attribute__((always_inline)) {
    const int b = plan.off[lw.slot] + lw.chunk * RC;
    const int n = plan.off[lw.slot + 1] - b;
    const int c = UP ? r16 : (r16 & 7);
    bvo = kPastBuffer;
    if (c < n) {
      const int p = plan.order[b + c];
      bvo = (UP ? p / a.top_k : (r16 >> 3) * pairs + p) * K * 2 + 32 * grp;
    }
  };
  auto set_tile = [&]() __attribute__((always_inline)) {
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[lw.slot]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rb = UP ? lw.tile + i * tiles : 2 * lw.tile + i;
      const size_t t0 = (size_t)rb * KBT + kb0;
      wrs[i] = __builtin_amdgcn_make_buffer_rsrc((void*)(w + e * wbytes + t0 * 2048), (short)0,
                                                 nbw * 2048, kBufferWord3);
      srs[i] = __builtin_amdgcn_make_buffer_rsrc((void*)(ws + e * wsbytes + t0 * 64), (short)0,
                                                 nbw * 64, kBufferWord3);
    }
  };
  set_rows();
  set_tile();
  v4u wlo[D][2], whi[D][2], bx[D][4];
  uint32_t wsc[D][2];
  // One K block into ring slot d; past the run's end the offsets lie past the
  // buffers (zeros, no memory access), so every step issues the same loads.
  auto load = [&](int d) __attribute__((always_inline)) {
    const int vo = live ? 16 * lane : kPastBuffer;
    const int so = live ? 4 * r16 : kPastBuffer;
    const int bo = live ? bvo : kPastBuffer;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wlo[d][i] = __builtin_amdgcn_raw_buffer_load_b128(wrs[i], vo, lkb * 2048, kLoadNontemporal);
      whi[d][i] =
          __builtin_amdgcn_raw_buffer_load_b128(wrs[i], vo + 1024, lkb * 2048, kLoadNontemporal);
      wsc[d][i] = __builtin_amdgcn_raw_buffer_load_b32(srs[i], so, lkb * 64, 0);
    }
    const int bk = (kb0 + lkb) * 256;
    bx[d][0] = __builtin_amdgcn_raw_buffer_load_b128(brs, bo, bk, 0);
    bx[d][1] = __builtin_amdgcn_raw_buffer_load_b128(brs, bo + 16, bk, 0);
    bx[d][2] = __builtin_amdgcn_raw_buffer_load_b128(brs, bo + 128, bk, 0);
    bx[d][3] = __builtin_amdgcn_raw_buffer_load_b128(brs, bo + 144, bk, 0);
    if (live && ++lkb == nbw) {
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
  cw.start(plan, item0, tiles);
  int64_t citem = item0;
  int ckb = 0, buf = 0;
  v4f acc[2] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
  const int sb0 = grp >> 1;  // 32-block of this lane's first 16 K (its second is sb0 + 2)
  auto consume = [&](int d) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f0 = e8m0_to_f32((wsc[d][i] >> (8 * sb0)) & 0xFFu);
      const float f1 = e8m0_to_f32((wsc[d][i] >> (8 * (sb0 + 2))) & 0xFFu);
      const v8bf a0 = fp8x8_to_bf16(wlo[d][i].x, wlo[d][i].y, f0);
      const v8bf a1 = fp8x8_to_bf16(wlo[d][i].z, wlo[d][i].w, f0);
      const v8bf a2 = fp8x8_to_bf16(whi[d][i].x, whi[d][i].y, f1);
      const v8bf a3 = fp8x8_to_bf16(whi[d][i].z, whi[d][i].w, f1);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, __builtin_bit_cast(v8bf, bx[d][0]),
                                                       acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, __builtin_bit_cast(v8bf, bx[d][1]),
                                                       acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a2, __builtin_bit_cast(v8bf, bx[d][2]),
                                                       acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a3, __builtin_bit_cast(v8bf, bx[d][3]),
                                                       acc[i], 0, 0, 0);
    }
  };
  // The item's partial tiles -> LDS (two buffers in turn: a wave writes one
  // again only after the barrier of the item between, which every wave reaches
  // after reading it), their sum in ascending K order, the epilogue.
  auto finish = [&]() __attribute__((always_inline)) {
    const int b = __builtin_amdgcn_readfirstlane(plan.off[cw.slot]) + cw.chunk * RC;
    int n = __builtin_amdgcn_readfirstlane(plan.off[cw.slot + 1]) - b;
    n = n < RC ? n : RC;
    if ((UP ? r16 : (r16 & 7)) < n) {
      float* q = &red[buf][wave][r16 * kColStride + 4 * grp];
      *reinterpret_cast<v4f*>(q) = acc[0];
      *reinterpret_cast<v4f*>(q + 16) = acc[1];
    }
    acc[0] = acc[1] = v4f{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    if constexpr (UP) {
      const int col = tid >> 4, row = tid & 15;
      if (col < n) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          g += red[buf][v][col * kColStride + row];
          u += red[buf][v][col * kColStride + 16 + row];
        }
        const float h = g / (1.f + expf(-g)) * u;
        const __bf16 hi = (__bf16)h;
        // A high part beyond BF16's range has no remainder.
        const __bf16 lo = fabsf((float)hi) < INFINITY ? (__bf16)(h - (float)hi) : (__bf16)0.f;
        const size_t at = (size_t)plan.order[b + col] * a.inter + 16 * cw.tile + row;
        a.h[at] = __builtin_bit_cast(uint16_t, hi);
        a.h[(size_t)pairs * a.inter + at] = __builtin_bit_cast(uint16_t, lo);
      }
    } else {
      const int col = tid >> 5, row = tid & 31;
      if (col < n) {
        float y = 0.f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
          y += red[buf][v][col * kColStride + row] + red[buf][v][(col + 8) * kColStride + row];
        a.y[(size_t)plan.order[b + col] * a.hidden + 32 * cw.tile + row] = y;
      }
    }
    buf ^= 1;
    if (++citem < item1) cw.next(plan, tiles);
  };

  if (nbw == 0) {  // fewer K blocks than waves: this one adds zeros
    while (citem < item1) finish();
    return;
  }
#pragma unroll
  for (int d = 0; d < D; ++d) load(d);
  while (citem < item1) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (citem < item1) {
        consume(d);
        if (++ckb == nbw) {
          ckb = 0;
          finish();
        }
      }
      load(d);
    }
  }
}

// out[t] = sum_j weights[t, j] y[t, j], one thread per 8 columns.
__global__ void combine_kernel(ExpertArgs a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int cols = a.hidden >> 3;
  if (i >= (int64_t)a.tokens * cols) return;
  const int t = (int)(i / cols);
  const int c = (int)(i - (int64_t)t * cols);
  float s[8] = {};
  for (int j = 0; j < a.top_k; ++j) {
    const int p = t * a.top_k + j;
    if ((unsigned)a.ids[p] >= (unsigned)a.experts) continue;
    const float w = a.weights[p];
    const float4* y = reinterpret_cast<const float4*>(a.y + (size_t)p * a.hidden + 8 * c);
    const float4 y0 = y[0], y1 = y[1];
    s[0] = fmaf(w, y0.x, s[0]);
    s[1] = fmaf(w, y0.y, s[1]);
    s[2] = fmaf(w, y0.z, s[2]);
    s[3] = fmaf(w, y0.w, s[3]);
    s[4] = fmaf(w, y1.x, s[4]);
    s[5] = fmaf(w, y1.y, s[5]);
    s[6] = fmaf(w, y1.z, s[6]);
    s[7] = fmaf(w, y1.w, s[7]);
  }
  const uint4 v = {bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]), bf16_pair(s[4], s[5]),
                   bf16_pair(s[6], s[7])};
  *reinterpret_cast<uint4*>(a.out + (size_t)t * a.hidden + 8 * c) = v;
}

}  // namespace

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess)
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  // One workgroup per CU, never more than there can be items.
  const int64_t pairs = (int64_t)a.tokens * a.top_k;
  auto grid = [&](int64_t tiles) {
    const int64_t most = pairs * tiles;
    return dim3((unsigned)(most < cus ? most : cus));
  };
  hipLaunchKernelGGL((experts_kernel<true, 4>), grid(a.inter >> 4), dim3(kThreads), 0, s, a);
  hipLaunchKernelGGL((experts_kernel<false, 4>), grid(a.hidden >> 5), dim3(kThreads), 0, s, a);
  const int64_t work = (int64_t)a.tokens * (a.hidden >> 3);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((work + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mxg
