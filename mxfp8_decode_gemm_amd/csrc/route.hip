// Expert routing (gfx950): mxmoe_route of include/mxdecode.h.
//
// One wave per row. Lane l holds the logits of V neighbouring experts in
// registers, so a row is read once, in wide loads, and everything after it is
// cross-lane work:
//   * score s = softmax or sigmoid, choice c = s + bias;
//   * group scores (with groups), the kept groups as one 64-bit lane mask;
//   * top_k rounds of a wave-wide maximum of c, each taking the lowest index
//     among equals, the chosen one struck out.
// Choices are compared as FP64 values: among thousands of rows, two FP32 choices
// (a rounded sum of a rounded exponential) do fall on the wrong side of each
// other. Where the choice has the order of the logits themselves (no bias, and
// no sum of two in a group score) the FP32 logits decide, unless the row has
// logits whose FP64 scores may be equal; otherwise FP32 choices do where all that
// matter lie further apart than their error. The other rows are done in FP64
// (8 of 256 experts, grouped sigmoid with a bias: one row in 75).
// The weights are FP32, from FP64 scores where FP32 would lose them.

#include <hip/hip_runtime.h>

#include <type_traits>

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

// The sum of the wave, uniform.
__device__ __forceinline__ float wave_sum(float x) {
#define MXG_DPP_ADD(C, MASK)                                                               \
  x += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), C, \
                                                             MASK, 0xF, true))
  MXG_DPP_ADD(0x111, 0xF);
  MXG_DPP_ADD(0x112, 0xF);
  MXG_DPP_ADD(0x114, 0xF);
  MXG_DPP_ADD(0x118, 0xF);
  MXG_DPP_ADD(0x142, 0xA);
  MXG_DPP_ADD(0x143, 0xC);
#undef MXG_DPP_ADD
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
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

// Scores below FP64's normal range count as zero.
constexpr double kLeast = 0x1p-1022;
// FP64 decides at once where FP64 scores of different logits may come out equal
// (or in the other order). Where logits alone order the experts (by_logit):
//   softmax: exp(l - top) / sum has its argument rounded by 2^-53 |l - top|, exp
//   and quotient by 2^-51, relative; scores of logits that lie d apart differ
//   by d. FP32 neighbours lie |l| 2^-24 and more apart: four times the error
//   of both scores where |l| >= 2^-26 (|top| + 4);
//   sigmoid: exp, sum and reciprocal are off by 2^-51, relative; scores of logits that
//   lie d apart differ by d (1 - s) >= d exp(-max(l, 0)) / 2 at the larger l. FP32
//   neighbours below kNearOneByLogit (2^-19 exp(-18) / 2 at 18) and with
//   |l| >= 2^-22 are 2^-47 and more apart by that measure.
// Both hold above kNearZero (|top| + 16), with top = 0 for the sigmoid.
// With a bias or sums of two, sigmoids above kNearOne are one but for 2^-43.
constexpr float kNearZero = 0x1p-26f;
constexpr float kNearOneByLogit = 18.f;
constexpr float kNearOne = 30.f;

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// What the lanes of a row's wave hold: lane l the experts V l .. V l + V - 1, so
// that a row is read in wide loads and the lowest index of equals is the first
// lane's.
template <int V>
struct Row {
  float l[V];  // the logits; -infinity: out
  float top, inv;  // softmax: the largest, 1 / sum of the terms
};

// The sum of the softmax's terms, uniform (0: every expert is out).
template <int V>
__device__ __forceinline__ double score_sum64(const Row<V>& row) {
  double sum = 0.0;
  if (row.top > -INFINITY) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += soft_term<double>(row.l[i], row.top);
  }
  return wave_sum(sum);
}

// Chooses in FP64: lane j gets the expert of place j (-1: none).
template <int V>
__device__ __forceinline__ int choose_wide(const RouteArgs& a, const Row<V>& row,
                                                     double* cs, int lane) {
  const int E = a.r.experts, G = a.r.groups, per = E / G;
  const bool softmax = a.r.score == MXG_ROUTE_SOFTMAX;
  double c[V];
  const double sum = softmax ? score_sum64<V>(row) : 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float l = row.l[i];
    double s = -INFINITY;
    if (l > -INFINITY) {
      s = softmax ? soft_term<double>(l, row.top) / sum : sigmoid64(l);
      if (s < kLeast) s = 0.0;
      if (a.bias) s += (double)a.bias[V * lane + i];
      if (!(s > -INFINITY)) s = -INFINITY;  // a NaN bias: out
    }
    c[i] = s;
  }
  if (G > 1 && a.r.top_groups < G) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (V * lane + i < E) cs[V * lane + i] = c[i];
    __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
    double score = -INFINITY;         // lane g: of group g
    if (lane < G) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int q = lane * per; q < (lane + 1) * per; ++q) {
        const double v = cs[q];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      score = a.r.group_best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
    int ahead = 0;  // groups before this one
    for (int g = 0; g < G; ++g) {
      const double o = lane_f64(score, g);
      ahead += o > score || (o == score && g < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < G && ahead < a.r.top_groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = V * lane + i;
      if (e < E && !((kept >> (e / per)) & 1)) c[i] = -INFINITY;
    }
  }
  int id = -1;
  for (int j = 0; j < a.r.top_k; ++j) {
    double best = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = fmax(best, c[i]);
    const double m = wave_max(best);
    if (!(m > -INFINITY)) break;  // nothing left
    const int who = __ffsll((unsigned long long)__ballot(best == m)) - 1;
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (c[i] == m) at = i;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane == who && at == i) c[i] = -INFINITY;
    at = __builtin_amdgcn_readlane(at, who);
    if (lane == j) id = V * who + at;
  }
  return id;
}

// Chosen scores of logits further than this below the largest (softmax), or
// below zero (sigmoid), make their row's weights in FP64. The others are at least
// exp(-64) / 1024 and keep all their bits in FP32.
constexpr float kSmall = 64.f;

// The weight of this lane's choice (id < 0: none) from FP64 scores: their ratios
// and their products with the scale hold where FP32 scores would be subnormal or
// zero. One rounding to FP32.
template <int V>
__device__ __forceinline__ float wide_weight(const RouteArgs& a, const Row<V>& row, int id,
                                             float logit) {
  double s = 0.0;
  if (a.r.score == MXG_ROUTE_SOFTMAX) {
    const double sum = score_sum64<V>(row);
    if (id >= 0) s = soft_term<double>(logit, row.top) / sum;
  } else if (id >= 0) {
    s = sigmoid64(logit);
  }
  if (s < kLeast) s = 0.0;
  if (a.r.renormalize) {
    const double sum = wave_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  return (float)(s * (double)a.r.scale);
}

// ---- FP32 choices, where they decide ---------------------------------------
// Either the logits themselves (exact), or choices with an error below
// 2^-19 (1 + |c|), given up where two that matter lie closer than kTol:
//   sigmoid: 1 / (1 + e), e = 2^(-l log2 e) to 1.5 |l| 2^-24 + 2^-22 relative,
//   moves s by at most s (1 - s) of that, s (1 - s) |l| < 0.23; softmax: the
//   term the same with s |d| < 0.37, the sum's 22 roundings; one reciprocal; the
//   sum with the bias. A group's score adds two: its error is below
//   2^-18 (1 + |c1| + |c2|), however small the sum.
constexpr float kTol = 0x1p-17f;

// Floats as integers of the same order (negative zero just below zero).
__device__ __forceinline__ int key_of(float x) {
  const int b = (int)__float_as_uint(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_key(int k) {
  return __uint_as_float((uint32_t)(k ^ ((k >> 31) & 0x7FFFFFFF)));
}
constexpr int kOut = (int)0x80000000;  // below every key

// The largest x of the wave, uniform.
__device__ __forceinline__ int wave_max(int x) {
#define MXG_DPP_MAX(C, MASK) \
  x = max(x, __builtin_amdgcn_update_dpp(kOut, x, C, MASK, 0xF, false))
  MXG_DPP_MAX(0x111, 0xF);
  MXG_DPP_MAX(0x112, 0xF);
  MXG_DPP_MAX(0x114, 0xF);
  MXG_DPP_MAX(0x118, 0xF);
  MXG_DPP_MAX(0x142, 0xA);
  MXG_DPP_MAX(0x143, 0xC);
#undef MXG_DPP_MAX
  return __builtin_amdgcn_readlane(x, 63);
}

// exp(x) to 1.5 |x| 2^-24 + 2^-22 relative.
__device__ __forceinline__ float exp_near(float x) {
  return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// A lane's two largest keys and their places; of equals the lower place first.
struct Two {
  int b1 = kOut, b2 = kOut, a1 = 0, a2 = 0;

  __device__ __forceinline__ void add(int k, int place) {
    const bool first = k > b1, second = k > b2;
    b2 = first ? b1 : (second ? k : b2);
    a2 = first ? a1 : (second ? place : a2);
    b1 = first ? k : b1;
    a1 = first ? place : a1;
  }
  // The two largest of this and another lane's (places are not kept).
  __device__ __forceinline__ void merge(int o1, int o2) {
    b2 = max(max(b2, o2), min(b1, o1));
    b1 = max(b1, o1);
  }
};

template <int C>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, C, 0xF, 0xF, false);
}

// The two largest of the 2^log lanes around, in each of them.
__device__ __forceinline__ Two around(Two t, int log) {
  if (log > 0) t.merge(dpp<0xB1>(t.b1), dpp<0xB1>(t.b2));    // lane ^ 1
  if (log > 1) t.merge(dpp<0x4E>(t.b1), dpp<0x4E>(t.b2));    // lane ^ 2
  if (log > 2) t.merge(dpp<0x141>(t.b1), dpp<0x141>(t.b2));  // the other quad of 8
  if (log > 3) t.merge(dpp<0x140>(t.b1), dpp<0x140>(t.b2));  // the other 8 of 16
  for (int o = 16; o < 1 << log; o <<= 1)
    t.merge(__shfl_xor(t.b1, o, 64), __shfl_xor(t.b2, o, 64));
  return t;
}

// Whether the choices have the order of the logits.
__device__ __forceinline__ bool ordered_by_logit(const RouteArgs& a) {
  return !a.bias && (a.r.groups == 1 || a.r.group_best == 1 || a.r.experts == a.r.groups);
}

// Lane j gets the expert of place j in *id; false: FP64 has to decide.
template <int V>
__device__ __forceinline__ bool choose(const RouteArgs& a, const Row<V>& row, int* cs, int lane,
                                       int* id) {
  const int E = a.r.experts, G = a.r.groups, per = E / G;
  const bool softmax = a.r.score == MXG_ROUTE_SOFTMAX;
  const bool by_logit = ordered_by_logit(a);
  int k[V];  // the choices' keys
  Two two;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float c = row.l[i];
    if (!by_logit) {
      c = softmax ? exp_near(c - row.top) * row.inv
                  : __builtin_amdgcn_rcpf(1.f + exp_near(-c));
      if (a.bias) c += a.bias[V * lane + i < E ? V * lane + i : 0];
    }
    // (Negative zero becomes zero. A NaN bias: out.)
    k[i] = row.l[i] > -INFINITY && c > -INFINITY ? key_of(c + 0.f) : kOut;
    two.add(k[i], i);
  }
  if (G > 1 && a.r.top_groups < G) {
    // The 2^log lanes of a group hold its experts (aligned), or else scan its
    // choices in LDS; their two largest make its score.
    const int log = a.group_log, g = lane >> log, sub = lane & ((1 << log) - 1);
    Two best = two;
    if (!a.aligned) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (V * lane + i < E) cs[V * lane + i] = k[i];
      __builtin_amdgcn_wave_barrier();  // LDS is in order within the wave
      best = Two();
      if (g < G)
        for (int q = sub; q < per; q += 1 << log) best.merge(cs[g * per + q], kOut);
    }
    best = around(best, log);
    float score = best.b1 == kOut ? -INFINITY : of_key(best.b1);
    float size = fabsf(score);  // of what the score is a sum of: its error's measure
    if (a.r.group_best == 2 && best.b2 != kOut) {
      size += fabsf(of_key(best.b2));
      score += of_key(best.b2);
    }
    // Lane sub of a group compares it with groups sub, sub + 2^log, ...
    const uint64_t mine = (log == 6 ? ~0ull : (1ull << (1 << log)) - 1) << (g << log);
    int ahead = 0;  // groups before this one
    bool close = false;
    for (int h0 = 0; h0 < G; h0 += 1 << log) {
      const int h = h0 + sub;
      const float o = __shfl(score, (h < G ? h : 0) << log, 64);
      const bool other = h < G && h != g;
      ahead += __popcll(__ballot(other && (o > score || (o == score && h < g))) & mine);
      if (!by_logit) {
        // (Of two groups each compares with the other, by its own size.)
        close |= other && g < G && o > -INFINITY && score > -INFINITY &&
                 !(fabsf(o - score) > 2 * kTol * (1.f + size));
      }
    }
    if (__any(close)) return false;
    if (a.aligned) {
      const bool out = ahead >= a.r.top_groups;
#pragma unroll
      for (int i = 0; i < V; ++i) k[i] = out ? kOut : k[i];
      two.b1 = out ? kOut : two.b1;
      two.b2 = out ? kOut : two.b2;
    } else {
      const uint64_t kept = __ballot(ahead < a.r.top_groups);
      two = Two();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int of = (int)(((uint32_t)(V * lane + i) * a.per_inv) >> 20);  // its group
        if (!((kept >> (of << log)) & 1)) k[i] = kOut;
        two.add(k[i], i);
      }
    }
  }
  // Rounds of the largest: the lowest lane that has it gives up its first. A
  // lane that has given both looks again at all it holds (seldom).
  int out = -1, key = kOut, n = 0;
  uint64_t gave = 0;  // lanes whose first of two is gone
  const int rounds = by_logit ? a.r.top_k : a.r.top_k + 1;
  for (; n < rounds; ++n) {
    const int m = wave_max(two.b1);
    if (m == kOut) break;  // nothing left
    const uint64_t has = __ballot(two.b1 == m);
    const int who = __ffsll((unsigned long long)has) - 1;
    const int place = __builtin_amdgcn_readlane(two.a1, who);
    out = lane == n ? V * who + place : out;
    key = lane == n ? m : key;
    if (lane == who) {
      two.b1 = two.b2;
      two.a1 = two.a2;
      two.b2 = kOut;
    }
    if constexpr (V > 2) {
      if ((gave >> who) & 1) {
        if (lane == who) {
          two = Two();
#pragma unroll
          for (int i = 0; i < V; ++i)
            two.add(k[i] < m || (k[i] == m && i > place) ? k[i] : kOut, i);
        }
        gave &= ~(1ull << who);
      } else {
        gave |= 1ull << who;
      }
    }
  }
  if (!by_logit) {  // neighbours in the order lie apart (one round more than top_k)
    const float c = of_key(key), before = __shfl_up(c, 1, 64);
    if (__any(lane > 0 && lane < n && !(before - c > kTol * (1.f + fabsf(c))))) return false;
  }
  *id = lane < a.r.top_k ? out : -1;
  return true;
}

template <int V, bool BF16>
__global__ void __launch_bounds__(64 * kWaves) route_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kWaves + wave;
  if (t >= a.tokens) return;  // whole waves; no barrier below
  const int E = a.r.experts;
  const bool softmax = a.r.score == MXG_ROUTE_SOFTMAX;

  Row<V> row;
  using Raw = std::conditional_t<BF16, uint16_t, uint32_t>;
  const Raw* src = reinterpret_cast<const Raw*>(a.logits) + (int64_t)t * a.row_stride;
  Raw raw[V];
  struct alignas(sizeof(Raw) * V) Wide { Raw v[V]; };
  if (E % V == 0 && (reinterpret_cast<uintptr_t>(src) & (sizeof(Wide) - 1)) == 0) {
    if (V * lane < E) *reinterpret_cast<Wide*>(raw) = reinterpret_cast<const Wide*>(src)[lane];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (V * lane + i < E) raw[i] = src[V * lane + i];
  }
  float hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = -INFINITY;
    if (V * lane + i < E) v = __uint_as_float(BF16 ? (uint32_t)raw[i] << 16 : (uint32_t)raw[i]);
    row.l[i] = v > -INFINITY ? v : -INFINITY;  // NaN: out
    hi = fmaxf(hi, row.l[i]);
  }
  row.top = 0.f;
  row.inv = 0.f;
  if (softmax) {
    row.top = hi = of_key(wave_max(key_of(hi)));
    float sum = 0.f;
    if (hi > -INFINITY) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += soft_term<float>(row.l[i], hi);
    }
    sum = wave_sum(sum);
    row.inv = sum > 0.f ? 1.f / sum : 0.f;
  }

  // FP32 first; FP64 for rows with choices too close to each other, or with
  // scores that are about one, or zero, in FP64.
  uint8_t* const cs = lds + sizeof(double) * (size_t)wave * E;
  const bool by_logit = ordered_by_logit(a);
  const float zero = by_logit ? kNearZero * (fabsf(row.top) + 16.f) : 0.f;
  bool odd = softmax ? hi == INFINITY : hi > (by_logit ? kNearOneByLogit : kNearOne);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    odd |= row.l[i] > -INFINITY && row.l[i] < (softmax ? hi : 0.f) - 700.f;
    odd |= fabsf(row.l[i]) < zero && row.l[i] != 0.f;
  }
  int id = -1;
  if (__any(odd) || !choose<V>(a, row, reinterpret_cast<int*>(cs), lane, &id))
    id = choose_wide<V>(a, row, reinterpret_cast<double*>(cs), lane);
  float logit = -INFINITY;
  if (id >= 0) logit = BF16 ? __uint_as_float((uint32_t)src[id] << 16) : __uint_as_float(src[id]);

  float w = 0.f;
  if (__builtin_expect(__any(id >= 0 && logit < (softmax ? row.top : 0.f) - kSmall), 0)) {
    w = wide_weight<V>(a, row, id, logit);
  } else {
    if (id >= 0)
      w = softmax ? soft_term<float>(logit, row.top) * row.inv : 1.f / (1.f + expf(-logit));
    if (a.r.renormalize) {
      const float sum = wave_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    }
    w *= a.r.scale;
  }
  if (lane < a.r.top_k) {
    const int64_t at = (int64_t)t * a.r.top_k + lane;
    a.ids[at] = id;
    a.weights[at] = id >= 0 ? w : 0.f;
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

hipError_t launch_route(const RouteArgs& args, int logits_type, hipStream_t s) {
  RouteArgs a = args;
  const int per = a.r.experts / a.r.groups;
  a.per_inv = ((1u << 20) + per - 1) / per;  // exact for e < 1024, per <= 1024
  a.group_log = 6;
  while ((a.r.groups << a.group_log) > 64) --a.group_log;
  // Where a group fills 2^i whole lanes, these are its lanes.
  int v = 1;
  while (64 * v < a.r.experts) v *= 2;
  const int lanes = per / v;
  a.aligned = per % v == 0 && (lanes & (lanes - 1)) == 0;
  if (a.aligned)
    for (a.group_log = 0; 1 << a.group_log < lanes;) ++a.group_log;
  if (logits_type == MXG_BF16)
    launch<true>(a, s);
  else
    launch<false>(a, s);
  return hipGetLastError();
}

}  // namespace mxg
