// Expert routing (gfx950): mxmoe_route of include/mxdecode.h.
//
// One wave per row. Lane l holds the logits of experts l, l + 64, ... in
// registers (V of them), so a row is read once, coalesced, and everything
// after it is cross-lane work:
//   * score s = softmax or sigmoid, choice c = s + bias;
//   * group scores (with groups), the kept groups as one 64-bit lane mask;
//   * top_k rounds of a wave-wide maximum of c, each taking the lowest index
//     among equals, the chosen one struck out.
// Choices are compared in FP64: among thousands of rows, two FP32 choices
// (a rounded sum of a rounded exponential) do fall on the wrong side of each
// other. Where the choice has the order of the logits themselves (no bias,
// and no sum of two in a group score), the logits are compared instead and no
// FP64 exponential is taken, except above kNearOne. The weights are FP32.

#include <hip/hip_runtime.h>

#include "mxdecode_internal.h"

namespace mxg {
namespace {

constexpr int kWaves = 4;  // rows per workgroup

// x of the lane that DPP control C names (x itself where there is none).
template <int C>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, C, 0xF, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, C, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)l | ((uint64_t)h << 32));
}

__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)l | ((uint64_t)h << 32));
}

// The largest x of the wave, in every lane (no NaN among them): row shifts by
// 1, 2, 4 and 8, then the row broadcasts; lane 63 holds the maximum.
__device__ __forceinline__ double wave_max(double x) {
  x = fmax(x, dpp_f64<0x111>(x));
  x = fmax(x, dpp_f64<0x112>(x));
  x = fmax(x, dpp_f64<0x114>(x));
  x = fmax(x, dpp_f64<0x118>(x));
  x = fmax(x, dpp_f64<0x142>(x));
  x = fmax(x, dpp_f64<0x143>(x));
  return lane_f64(x, 63);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// exp(l - m) of a softmax whose largest logit is m (m = +infinity: 1 for the
// logits that are +infinity, else 0). l = -infinity gives 0.
template <typename F>
__device__ __forceinline__ F soft_term(float l, float m) {
  if (m == INFINITY) return l == INFINITY ? F(1) : F(0);
  if constexpr (sizeof(F) == 8)
    return exp((double)l - (double)m);
  else
    return expf(l - m);
}

// Scores below FP64's normal range count as zero: those of logits this far
// below the largest (softmax) or below zero (sigmoid).
constexpr double kZeroBelow = -708.3964185322641;  // ln 2^-1022
constexpr double kLeast = 0x1p-1022;
// From here on neighbouring logits can have the same FP64 sigmoid.
constexpr float kNearOne = 30.f;

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// A value in the order of the sigmoids' FP64 values, equal where they are. The
// scores above kNearOne differ by multiples of 2^-53 up to 2^-43, so
// 30 + 2^46 times their difference from sigmoid(30) is exact.
__device__ __forceinline__ double sigmoid_order(float l) {
  if (l > kNearOne) return kNearOne + 0x1p46 * (sigmoid64(l) - sigmoid64(kNearOne));
  return l > (float)kZeroBelow ? (double)l : kZeroBelow;
}

template <int V, bool BF16>
__global__ void __launch_bounds__(64 * kWaves) route_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = blockIdx.x * kWaves + wave;
  if (row >= a.tokens) return;  // whole waves; no barrier below
  const int E = a.r.experts;
  const bool softmax = a.r.score == MXG_ROUTE_SOFTMAX;
  const int per = E / a.r.groups;

  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    float v = -INFINITY;
    if (e < E) {
      const int64_t at = (int64_t)row * a.row_stride + e;
      if constexpr (BF16)
        v = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(a.logits)[at] << 16);
      else
        v = reinterpret_cast<const float*>(a.logits)[at];
    }
    l[i] = v > -INFINITY ? v : -INFINITY;  // NaN: out
  }

  // Softmax: the largest logit and the sum of the terms.
  float top = 0.f, inv = 0.f;
  if (softmax) {
    double m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmax(m, (double)l[i]);
    top = (float)wave_max(m);
    float sum = 0.f;
    if (top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += soft_term<float>(l[i], top);
    }
    sum = wave_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }

  // The choices.
  double c[V];
  const bool by_logit = !a.bias && (a.r.groups == 1 || a.r.group_best == 1 || per == 1);
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = -INFINITY;
      if (l[i] > -INFINITY) {
        if (softmax)  // (the difference is NaN where both are +infinity)
          c[i] = l[i] == top ? 0.0 : fmax((double)l[i] - (double)top, kZeroBelow);
        else
          c[i] = sigmoid_order(l[i]);
      }
    }
  } else {
    double inv64 = 1.0;
    if (softmax) {
      double sum = 0.0;
      if (top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum += soft_term<double>(l[i], top);
      }
      sum = wave_sum(sum);
      inv64 = sum > 0.0 ? 1.0 / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      double s = -INFINITY;
      if (l[i] > -INFINITY) {
        s = softmax ? soft_term<double>(l[i], top) * inv64 : sigmoid64(l[i]);
        if (s < kLeast) s = 0.0;
        if (a.bias) s += (double)a.bias[e];
        if (!(s > -INFINITY)) s = -INFINITY;  // a NaN bias: out
      }
      c[i] = s;
    }
  }

  if (a.r.groups > 1 && a.r.top_groups < a.r.groups) {
    double* cs = reinterpret_cast<double*>(lds) + (size_t)wave * E;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 64 + lane < E) cs[i * 64 + lane] = c[i];
    __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
    // Lane g: the score of group g.
    double score = -INFINITY;
    if (lane < a.r.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int q = lane * per; q < (lane + 1) * per; ++q) {
        const double v = cs[q];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      score = a.r.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
    int ahead = 0;  // groups before this one
    for (int g = 0; g < a.r.groups; ++g) {
      const double s = lane_f64(score, g);
      ahead += s > score || (s == score && g < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.r.groups && ahead < a.r.top_groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (e < E && !((kept >> (e / per)) & 1)) c[i] = -INFINITY;
    }
  }

  // top_k rounds; lane j keeps the j-th expert and its logit.
  int id = -1;
  float logit = -INFINITY;
  for (int j = 0; j < a.r.top_k; ++j) {
    double m = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmax(m, c[i]);
    m = wave_max(m);
    if (!(m > -INFINITY)) break;  // nothing left
    bool found = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t eq = __ballot(c[i] == m);
      if (!found && eq) {
        found = true;
        const int who = __ffsll((unsigned long long)eq) - 1;
        const float li = __uint_as_float(
            (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(l[i]), who));
        if (lane == j) {
          id = i * 64 + who;
          logit = li;
        }
        if (lane == who) c[i] = -INFINITY;
      }
    }
  }
  float w = 0.f;
  if (id >= 0) w = softmax ? soft_term<float>(logit, top) * inv : 1.f / (1.f + expf(-logit));
  if (a.r.renormalize) {
    const float sum = wave_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < a.r.top_k) {
    const int64_t at = (int64_t)row * a.r.top_k + lane;
    a.ids[at] = id;
    a.weights[at] = id >= 0 ? w * a.r.scale : 0.f;
  }
}

template <bool BF16>
void launch(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + kWaves - 1) / kWaves)), block(64 * kWaves);
  const size_t lds = a.r.groups > 1 ? sizeof(double) * kWaves * a.r.experts : 0;
  const int v = (a.r.experts + 63) / 64;
  if (v <= 1)
    hipLaunchKernelGGL((route_kernel<1, BF16>), grid, block, lds, s, a);
  else if (v <= 2)
    hipLaunchKernelGGL((route_kernel<2, BF16>), grid, block, lds, s, a);
  else if (v <= 4)
    hipLaunchKernelGGL((route_kernel<4, BF16>), grid, block, lds, s, a);
  else if (v <= 8)
    hipLaunchKernelGGL((route_kernel<8, BF16>), grid, block, lds, s, a);
  else
    hipLaunchKernelGGL((route_kernel<16, BF16>), grid, block, lds, s, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int logits_type, hipStream_t s) {
  if (logits_type == MXG_BF16)
    launch<true>(a, s);
  else
    launch<false>(a, s);
  return hipGetLastError();
}

}  // namespace mxg
