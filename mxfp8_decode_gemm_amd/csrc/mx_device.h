// Device helpers shared by the kernels that stream MXFP8 weights (gfx950):
// vector types, the operand conversions, raw buffer constants, scope-marked
// loads and stores, BF16 packing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// 2^(s-127) as an FP32 multiplier: the biased exponent s in the exponent
// field; s == 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  // 2^-127 (an FP32 subnormal, kept: the library is built with FP32
  // denormals on) times 2^s, one instruction; s = 255 gives +inf.
  return __builtin_amdgcn_ldexpf(__uint_as_float(0x00400000u), (int)s);
}

// Eight e4m3fn bytes (two dwords, lowest byte first) times a power-of-two
// scale, as eight BF16 values. v_cvt_scalef32_pk_bf16_fp8 converts two bytes
// of a dword per instruction; an e4m3 value times 2^k is exact in BF16 for
// every scale the workloads use, and the instruction rounds to nearest even.
__device__ __forceinline__ v8bf fp8x8_to_bf16(uint32_t w0, uint32_t w1, float scale) {
  const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
  const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
  const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
  const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Raw buffer descriptors (gfx9 family): the fourth word of a plain byte
// buffer, an offset no descriptor here reaches (1 GiB; offsets at or past a
// buffer's size read as zeros), and the cache policy of a streaming load.
constexpr int kBufferWord3 = 0x00020000;
constexpr int kPastBuffer = 0x40000000;
constexpr int kLoadNontemporal = 2;

// A word that nothing writes while the kernel runs, read at a wave-uniform
// address through the constant address space: a scalar load, counted apart
// from the vector loads of the W stream, so a wait for it never waits for
// the stream (the dispatch's acquire makes earlier launches' stores visible).
__device__ __forceinline__ uint32_t ld_uniform_u32(const uint32_t* p) {
  return *(const __attribute__((address_space(4))) uint32_t*)(p);
}
// Lane i takes lane i + N of its 16-lane row (0 where that lies past the
// row): a DPP move on the vector unit instead of an LDS permute.
template <int N>
__device__ __forceinline__ uint32_t row_down(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x100 + N, 0xF, 0xF, true);
}
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
__device__ __forceinline__ uint32_t ld_agent_u32(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_agent_u32(uint32_t* p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t ld_agent_u64(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_agent_u64(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// BF16 bits of an FP32 value, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __bf16 a = (__bf16)lo;
  const __bf16 b = (__bf16)hi;
  return (uint32_t)__builtin_bit_cast(uint16_t, a) |
         ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

// Each BF16 half equal to 0x8000 (negative zero) becomes 0x0000.
__device__ __forceinline__ uint32_t clear_negative_zero(uint32_t w) {
  const uint32_t lo = (w & 0xFFFFu) == 0x8000u ? 0u : (w & 0xFFFFu);
  const uint32_t hi = (w >> 16) == 0x8000u ? 0u : (w & 0xFFFF0000u);
  return lo | hi;
}

}  // namespace
}  // namespace mxg
