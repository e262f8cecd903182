// MXFP4 (gfx950): mxfp4_quantize, mxfp4_dequantize and mxrows_pack_weight of
// include/mxrows.h.

#include <hip/hip_runtime.h>

#include "mx_device.h"
#include "quant_device.h"
#include "rows_internal.h"

namespace mxg {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values of a row as FP32 (not kept in the caches: 16384 rows of 8192
// BF16, quantized and back, 103 us; 137 kept).
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (TYPE == MXG_F32) {
    const v4f* q = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + at);
    const v4f a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const v4u a = __builtin_nontemporal_load(
        reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(p) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == MXG_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xFFFFu));
        v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
      }
    }
  }
}

// The scale byte of a block whose largest magnitude has these FP32 bits: with
// amax = (1 + f) 2^(E - 127), amax <= 6 2^e = 1.5 2^(e + 2) holds first at e = E -
// 129 where f <= 1/2 and at E - 128 otherwise; never below -127. Subnormal FP32
// magnitudes are below 6 2^-127.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax) {
  const int E = (int)(amax >> 23);
  if (E == 0xFF) return 0xFFu;
  const int s = E - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return (uint32_t)(s < 0 ? 0 : s);
}

// Codes and scale byte of a lane's 8 values; the 4 lanes of a block side by side.
// v_cvt_scalef32_pk_fp4_f32 divides by the scale (a power of two: exact) and rounds
// once, ties to even, for every finite block (|v / 2^e| <= 6).
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t* scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t sb = *scale = fp4_scale_byte(quad_max(amax));
  uint32_t codes = 0;
  if (sb == 0xFFu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= (7u | (__float_as_uint(v[i]) >> 28 & 8u)) << (4 * i);
  } else {
    const float s = e8m0_to_f32(sb);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[0], v[1], s, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2], v[3], s, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4], v[5], s, 2);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6], v[7], s, 3);
  }
  return codes;
}

// One lane per 8 values ("chunk"), kFlight chunks of a lane in flight. Bound by HBM: 2
// or 4 bytes read, 17/32 written per value (16384 rows of 8192 and back 103 us from BF16,
// 6.6 TB/s, 108 from FP16, 174 from FP32; 111 with eight chunks in flight). Rows without a
// gap are one long row (rows == 1); otherwise blockIdx.y counts the rows, each with
// workgroups of its own, most of whose lanes have nothing to do where it is short (16384
// rows, this launch alone, without a gap and with one: 8192 values 55 and 60 us, 4096 30
// and 37, 1024 9 and 26, 128 3 and 25).
constexpr int kFlight = 4;
template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    quantize4_kernel(const void* x, int64_t row_stride, int rows, int64_t chunks, uint8_t* xq,
                     uint8_t* xs) {
  const int64_t stride = (int64_t)gridDim.x * kThreads * kFlight;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    for (int64_t base = (int64_t)blockIdx.x * kThreads * kFlight; base < chunks; base += stride) {
      float v[kFlight][8];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {  // (past the end: the last chunk; chunks % 4 == 0)
        const int64_t c = base + j * kThreads + threadIdx.x;
        load8<TYPE>(x, row * row_stride + 8 * (c < chunks ? c : chunks - 1), v[j]);
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int64_t c = base + j * kThreads + threadIdx.x;
        uint32_t sb;
        const uint32_t codes = codes8(v[j], &sb);
        if (c < chunks) {
          const int64_t to = row * chunks + c;
          reinterpret_cast<uint32_t*>(xq)[to] = codes;
          if ((c & 3) == 0) xs[to >> 2] = (uint8_t)sb;
        }
      }
    }
  }
}

// One lane per 8 codes, kFlight in flight. The FP32 product of an E2M1 value and a
// power of two is exact up to FP32's range; the type's rounding follows.
template <int TYPE>
__global__ void __launch_bounds__(kThreads)
    dequantize4_kernel(const uint8_t* xq, const uint8_t* xs, int64_t chunks, void* y) {
  const int64_t stride = (int64_t)gridDim.x * kThreads * kFlight;
  for (int64_t base = (int64_t)blockIdx.x * kThreads * kFlight; base < chunks; base += stride) {
    uint32_t codes[kFlight], sb[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int64_t c = base + j * kThreads + threadIdx.x, cc = c < chunks ? c : chunks - 1;
      codes[j] = reinterpret_cast<const uint32_t*>(xq)[cc];
      sb[j] = xs[cc >> 2];
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int64_t c = base + j * kThreads + threadIdx.x;
      if (c >= chunks) break;
      const float s = sb[j] == 0xFFu ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(sb[j]);
      float v[8];
#define MXG_FP4_PAIR(I)                                                        \
  {                                                                            \
    const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[j], 1.f, I); \
    v[2 * I] = p[0] * s;                                                       \
    v[2 * I + 1] = p[1] * s;                                                   \
  }
      MXG_FP4_PAIR(0)
      MXG_FP4_PAIR(1)
      MXG_FP4_PAIR(2)
      MXG_FP4_PAIR(3)
#undef MXG_FP4_PAIR
      if constexpr (TYPE == MXG_F32) {
        float4* q = reinterpret_cast<float4*>(y) + 2 * c;
        q[0] = float4{v[0], v[1], v[2], v[3]};
        q[1] = float4{v[4], v[5], v[6], v[7]};
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (TYPE == MXG_BF16)
            w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
          else
            w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
        }
        reinterpret_cast<uint4*>(y)[c] = uint4{w[0], w[1], w[2], w[3]};
      }
    }
  }
}

// One thread per 16 bytes of the packed codes (the layout of rows_internal.h);
// K past the row's and rows past n are zeros.
template <int FORMAT>
__global__ void __launch_bounds__(kThreads)
    pack_codes_kernel(const uint8_t* w, int n, int k, int64_t pieces, int64_t per_expert,
                      uint4* wp) {
  constexpr int kUnit = FORMAT == MXG_MXFP4 ? 128 : 256;  // pieces of a unit
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int kbs = (int)(2 * ((k + 255) / 256));
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += stride) {
    const int64_t e = i / per_expert, u = (i - e * per_expert) / kUnit;
    const int in = (int)(i % kUnit), lane = in & 63, q = in >> 6;
    const int64_t rb = u / kbs;
    const int kb = (int)(u - rb * kbs), g = lane >> 5;
    const int64_t row = rb * 32 + (lane & 31);
    uint4 v = {0u, 0u, 0u, 0u};
    if (row < n && 128 * kb < k) {
      const int64_t r = e * n + row;
      if constexpr (FORMAT == MXG_MXFP4)  // q: the step
        v = *reinterpret_cast<const uint4*>(w + r * (k / 2) + 64 * kb + 16 * (2 * q + g));
      else                                // q: twice the step, the half
        v = *reinterpret_cast<const uint4*>(w + r * k + 128 * kb + 16 * (2 * q + g));
    }
    wp[i] = v;
  }
}

// One thread per scale word.
__global__ void __launch_bounds__(kThreads)
    pack_scales_kernel(const uint8_t* ws, int n, int k, int64_t words, int64_t per_expert,
                       uint32_t* wsp) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  const int kp = (k + 255) / 256;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += stride) {
    const int64_t e = i / per_expert, u = (i - e * per_expert) >> 6;
    const int lane = (int)(i & 63), g = lane >> 5;
    const int64_t rb = u / kp, row = rb * 32 + (lane & 31);
    const int kb = 2 * (int)(u - rb * kp);
    uint32_t v = 0x7F7F7F7Fu;
    if (row < n) {
      const uint8_t* p = ws + (e * n + row) * (k / 32) + 4 * kb + g;
      v = p[0] | (uint32_t)p[2] << 8;
      v |= 128 * (kb + 1) < k ? (uint32_t)p[4] << 16 | (uint32_t)p[6] << 24 : 0x7F7F0000u;
    }
    wsp[i] = v;
  }
}

unsigned blocks_for(int64_t threads) {
  const int64_t b = (threads + kThreads - 1) / kThreads;
  return (unsigned)(b < (1 << 20) ? b : 1 << 20);
}

}  // namespace

hipError_t launch_fp4_quantize(const void* x, int x_type, int64_t row_stride, int rows, int k,
                               uint8_t* xq, uint8_t* xs, hipStream_t s) {
  int64_t chunks = k / 8;
  if (row_stride == k) {
    chunks *= rows;
    rows = 1;
  }
  const dim3 grid(blocks_for((chunks + kFlight - 1) / kFlight),
                  (unsigned)(rows < 16384 ? rows : 16384)),
      block(kThreads);
  if (x_type == MXG_F32)
    hipLaunchKernelGGL((quantize4_kernel<MXG_F32>), grid, block, 0, s, x, row_stride, rows, chunks,
                       xq, xs);
  else if (x_type == MXG_BF16)
    hipLaunchKernelGGL((quantize4_kernel<MXG_BF16>), grid, block, 0, s, x, row_stride, rows, chunks,
                       xq, xs);
  else
    hipLaunchKernelGGL((quantize4_kernel<MXG_F16>), grid, block, 0, s, x, row_stride, rows, chunks,
                       xq, xs);
  return hipGetLastError();
}

hipError_t launch_fp4_dequantize(const uint8_t* xq, const uint8_t* xs, int rows, int k, int y_type,
                                 void* y, hipStream_t s) {
  const int64_t chunks = (int64_t)rows * (k / 8);
  const dim3 grid(blocks_for((chunks + kFlight - 1) / kFlight)), block(kThreads);
  if (y_type == MXG_F32)
    hipLaunchKernelGGL((dequantize4_kernel<MXG_F32>), grid, block, 0, s, xq, xs, chunks, y);
  else if (y_type == MXG_BF16)
    hipLaunchKernelGGL((dequantize4_kernel<MXG_BF16>), grid, block, 0, s, xq, xs, chunks, y);
  else
    hipLaunchKernelGGL((dequantize4_kernel<MXG_F16>), grid, block, 0, s, xq, xs, chunks, y);
  return hipGetLastError();
}

hipError_t launch_rows_pack(int format, const uint8_t* w, const uint8_t* ws, int experts, int n,
                            int k, uint8_t* wp, uint8_t* wsp, hipStream_t s) {
  const int64_t units = row_blocks(n) * kb_pairs(k) * 2;
  const int64_t per = units * unit_bytes(format) / 16, words = units / 2 * 64;
  const dim3 block(kThreads);
  if (format == MXG_MXFP4)
    hipLaunchKernelGGL((pack_codes_kernel<MXG_MXFP4>), dim3(blocks_for(per * experts)), block, 0, s,
                       w, n, k, per * experts, per, reinterpret_cast<uint4*>(wp));
  else
    hipLaunchKernelGGL((pack_codes_kernel<MXG_MXFP8>), dim3(blocks_for(per * experts)), block, 0, s,
                       w, n, k, per * experts, per, reinterpret_cast<uint4*>(wp));
  hipLaunchKernelGGL(pack_scales_kernel, dim3(blocks_for(words * experts)), block, 0, s, ws, n, k,
                     words * experts, words, reinterpret_cast<uint32_t*>(wsp));
  return hipGetLastError();
}

}  // namespace mxg
