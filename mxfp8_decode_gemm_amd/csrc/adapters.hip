// The first half of the rows' low-rank adapters (gfx950): u = scale A x, see
// mxgemm_lora in include/mxdecode.h. The second half, B u, is added in the
// GEMM's epilogue (gemm_kernel.h).

#include <hip/hip_runtime.h>

#include "mx_device.h"
#include "mxdecode_internal.h"

namespace mxg {
namespace {

constexpr int kWaves = 4;

// One wave per (row t, rank r): the row A[ids[t]][r] and x[t] in 8-value
// pieces per lane, FP32 sums.
__global__ void __launch_bounds__(64 * kWaves) shrink_kernel(ShrinkArgs a) {
  const int lane = threadIdx.x & 63;
  const int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= a.m * a.rank) return;
  const int t = item / a.rank, r = item - t * a.rank;
  const int i = a.ids[t];
  float s = 0.f;
  if ((unsigned)i < (unsigned)a.adapters) {
    const uint16_t* row = a.a + ((size_t)i * a.rank + r) * a.k;
    for (int k = 8 * lane; k < a.k; k += 512) {
      const uint4 av = *reinterpret_cast<const uint4*>(row + k);
      uint4 xv;
      if (a.xb) {
        xv = *reinterpret_cast<const uint4*>(a.xb + (size_t)t * a.k + k);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(a.x + (size_t)t * a.k + k);
        const uint32_t sb = a.xs[(size_t)t * (a.k >> 5) + (k >> 5)];
        xv = __builtin_bit_cast(uint4, fp8x8_to_bf16(c.x, c.y, e8m0_to_f32(sb)));
      }
      const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s = fmaf(__uint_as_float(aw[q] << 16), __uint_as_float(xw[q] << 16), s);
        s = fmaf(__uint_as_float(aw[q] & 0xFFFF0000u), __uint_as_float(xw[q] & 0xFFFF0000u), s);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    s *= a.scale[i];
  }
  if (lane == 0) a.u[item] = s;
}

}  // namespace

hipError_t launch_shrink(const ShrinkArgs& a, hipStream_t s) {
  const int items = a.m * a.rank;
  hipLaunchKernelGGL(shrink_kernel, dim3((unsigned)((items + kWaves - 1) / kWaves)),
                     dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace mxg
