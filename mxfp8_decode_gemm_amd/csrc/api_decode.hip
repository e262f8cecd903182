// C ABI of the per-row decode operators: host-side validation (from sizes and
// addresses only, before any HIP call) and dispatch. Declarations, argument
// meanings and error rules are in include/mxdecode.h.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/mxdecode.h"
#include "mxdecode_internal.h"
#include "mxgemm_internal.h"

using namespace mxg;

namespace {
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
int hip_code(hipError_t e) { return e == hipSuccess ? MXG_OK : MXG_EHIP; }

constexpr int32_t kMaxDim = 32768;  // of hidden and inter

bool expert_sizes_ok(int32_t tokens, int32_t top_k, int32_t experts, int32_t hidden,
                     int32_t inter) {
  return experts >= 1 && experts <= MXG_MOE_MAX_EXPERTS && tokens >= 1 && top_k >= 1 && (int64_t)tokens * top_k <= MXG_MOE_MAX_PAIRS && hidden > 0 &&
         hidden <= kMaxDim && hidden % 128 == 0 && inter > 0 && inter <= kMaxDim &&
         inter % 128 == 0;
}
}  // namespace

extern "C" {

int mxmoe_route(const mxmoe_router* r, const void* logits, int32_t logits_type,
                int64_t row_stride, const float* bias, int32_t tokens, int32_t* ids,
                float* weights, void* stream) {
  if (!r || !logits || !ids || !weights) return MXG_EINVAL;
  if (logits_type != MXG_F32 && logits_type != MXG_BF16) return MXG_EINVAL;
  if (r->experts < 1 || r->experts > MXG_ROUTE_MAX_EXPERTS) return MXG_EINVAL;
  if (r->score != MXG_ROUTE_SOFTMAX && r->score != MXG_ROUTE_SIGMOID) return MXG_EINVAL;
  if (r->groups < 1 || r->groups > MXG_ROUTE_MAX_GROUPS || r->experts % r->groups ||
      r->top_groups < 1 || r->top_groups > r->groups)
    return MXG_EINVAL;
  if (r->group_best != 1 && r->group_best != 2) return MXG_EINVAL;
  if (r->renormalize != 0 && r->renormalize != 1) return MXG_EINVAL;
  if (r->top_k < 1 || r->top_k > MXG_ROUTE_MAX_TOP_K ||
      r->top_k > r->experts / r->groups * r->top_groups)
    return MXG_EINVAL;
  if (tokens < 1 || tokens > (1 << 24) || row_stride < r->experts ||
      row_stride > ((int64_t)1 << 31))
    return MXG_EINVAL;
  if (!aligned(logits, logits_type == MXG_BF16 ? 2 : 4) || (bias && !aligned(bias, 4)) ||
      !aligned(ids, 4) || !aligned(weights, 4))
    return MXG_EALIGN;
  RouteArgs a;
  a.r = *r;
  a.logits = logits;
  a.row_stride = row_stride;
  a.bias = bias;
  a.tokens = tokens;
  a.ids = ids;
  a.weights = weights;
  return hip_code(launch_route(a, logits_type, static_cast<hipStream_t>(stream)));
}

size_t mxmoe_packed_weight_bytes(int32_t experts, int32_t n, int32_t k) {
  if (experts < 1 || experts > MXG_MOE_MAX_EXPERTS || n % 16) return 0;
  return (size_t)experts * mxgemm_packed_weight_bytes(n, k);
}

size_t mxmoe_packed_scale_bytes(int32_t experts, int32_t n, int32_t k) {
  if (experts < 1 || experts > MXG_MOE_MAX_EXPERTS || n % 16) return 0;
  return (size_t)experts * mxgemm_packed_scale_bytes(n, k);
}

int mxmoe_pack_weight(const uint8_t* w, const uint8_t* w_scale, int32_t experts, int32_t n,
                      int32_t k, uint8_t* w_packed, uint8_t* ws_packed, void* stream) {
  if (!w || !w_scale || !w_packed || !ws_packed) return MXG_EINVAL;
  if (mxmoe_packed_weight_bytes(experts, n, k) == 0) return MXG_EINVAL;
  if (!aligned16(w) || !aligned16(w_scale) || !aligned16(w_packed) || !aligned16(ws_packed))
    return MXG_EALIGN;
  return hip_code(launch_pack_weight(w, w_scale, n, k, w_packed, ws_packed,
                                     static_cast<hipStream_t>(stream), experts));
}

size_t mxmoe_workspace_bytes(int32_t tokens, int32_t top_k, int32_t experts, int32_t hidden,
                             int32_t inter) {
  if (!expert_sizes_ok(tokens, top_k, experts, hidden, inter)) return 0;
  ExpertArgs a = {};
  a.tokens = tokens;
  a.top_k = top_k;
  a.experts = experts;
  a.hidden = hidden;
  a.inter = inter;
  return experts_workspace(&a, nullptr);
}

int mxmoe_experts(const uint16_t* x, const int32_t* ids, const float* weights,
                  const uint8_t* w13, const uint8_t* w13_scale, const uint8_t* w2,
                  const uint8_t* w2_scale, int32_t tokens, int32_t top_k, int32_t experts,
                  int32_t hidden, int32_t inter, void* workspace, size_t workspace_bytes,
                  uint16_t* out, void* stream) {
  if (!x || !ids || !weights || !w13 || !w13_scale || !w2 || !w2_scale || !out) return MXG_EINVAL;
  if (!expert_sizes_ok(tokens, top_k, experts, hidden, inter)) return MXG_EINVAL;
  if (!aligned16(x) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned16(w13) ||
      !aligned16(w13_scale) || !aligned16(w2) || !aligned16(w2_scale) || !aligned16(out))
    return MXG_EALIGN;
  if (!workspace || workspace_bytes < mxmoe_workspace_bytes(tokens, top_k, experts, hidden, inter))
    return MXG_EWORKSPACE;
  if (!aligned16(workspace)) return MXG_EALIGN;
  ExpertArgs a;
  a.x = x;
  a.ids = ids;
  a.weights = weights;
  a.w13 = w13;
  a.w13s = w13_scale;
  a.w2 = w2;
  a.w2s = w2_scale;
  a.w13_bytes = mxgemm_packed_weight_bytes(2 * inter, hidden);
  a.w13s_bytes = mxgemm_packed_scale_bytes(2 * inter, hidden);
  a.w2_bytes = mxgemm_packed_weight_bytes(hidden, inter);
  a.w2s_bytes = mxgemm_packed_scale_bytes(hidden, inter);
  a.tokens = tokens;
  a.top_k = top_k;
  a.experts = experts;
  a.hidden = hidden;
  a.inter = inter;
  experts_workspace(&a, workspace);
  a.out = out;
  return hip_code(launch_experts(a, static_cast<hipStream_t>(stream)));
}

namespace {
// The scratch: header, one epoch word per workgroup, the pairs.
size_t lora_flag_bytes(int32_t n) {
  const size_t words = (size_t)(n + 15) / 16;  // tiles of at least 16 rows, or a split-K grid
  return (words < MXG_WS_MAX_GROUPS ? MXG_WS_MAX_GROUPS : (words + 3) / 4 * 4) * 4;
}
}  // namespace

size_t mxgemm_lora_scratch_bytes(int32_t n) {
  if (n <= 0 || n % 8) return 0;
  return MXG_WS_HEADER_BYTES + lora_flag_bytes(n) + kLoraMaxPairs * sizeof(uint64_t);
}

int mxgemm_lora_scratch_init(void* scratch, size_t scratch_bytes, void* stream) {
  if (!scratch || scratch_bytes < mxgemm_lora_scratch_bytes(8) || scratch_bytes % 16)
    return MXG_EINVAL;
  if (!aligned16(scratch)) return MXG_EALIGN;
  return hip_code(launch_workspace_init(static_cast<uint32_t*>(scratch), scratch_bytes,
                                        static_cast<hipStream_t>(stream)));
}

int mxgemm_lora(const mxg_mailbox* mb, const uint8_t* w, const uint8_t* w_scale,
                const uint8_t* x, const uint8_t* x_scale, const uint16_t* x_bf16, int32_t m,
                int32_t n, int32_t k, int32_t split_k, void* workspace, size_t workspace_bytes,
                const mxg_lora* lora, void* scratch, size_t scratch_bytes, uint16_t* c_out,
                void* stream) {
  if (!lora || !lora->a || !lora->b || !lora->scale || !lora->ids || lora->adapters < 1 ||
      lora->rank < 8 || lora->rank > MXG_LORA_MAX_RANK || lora->rank % 8)
    return MXG_EINVAL;
  const int rc = gemm_validate(mb, w, w_scale, x, x_scale, x_bf16, m, n, k, split_k, c_out,
                               nullptr, nullptr);
  if (rc != MXG_OK) return rc;
  if (!aligned16(lora->a) || !aligned16(lora->b) || !aligned(lora->scale, 4) ||
      !aligned(lora->ids, 4))
    return MXG_EALIGN;
  if (!scratch || scratch_bytes < mxgemm_lora_scratch_bytes(n)) return MXG_EWORKSPACE;
  if (!aligned16(scratch)) return MXG_EALIGN;
  uint8_t* s = static_cast<uint8_t*>(scratch);
  LoraArgs l = {};
  l.a = lora->a;
  l.b = lora->b;
  l.scale = lora->scale;
  l.ids = lora->ids;
  l.adapters = lora->adapters;
  l.rank = lora->rank;
  l.hdr = static_cast<uint32_t*>(scratch);
  // The pairs lie at one place for every n: a word that one call uses for a value
  // must not be another's flag.
  l.pairs = reinterpret_cast<uint64_t*>(s + MXG_WS_HEADER_BYTES);
  l.flags = reinterpret_cast<uint32_t*>(s + MXG_WS_HEADER_BYTES + kLoraMaxPairs * sizeof(uint64_t));
  return gemm_call(mb, w, w_scale, x, x_scale, x_bf16, m, n, k, split_k, workspace,
                   workspace_bytes, 0, c_out, nullptr, nullptr, stream, nullptr, nullptr, nullptr,
                   &l);
}

}  // extern "C"
