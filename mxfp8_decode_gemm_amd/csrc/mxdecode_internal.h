// Internal declarations of the per-row decode operators (routing, experts,
// adapters). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mxdecode.h"

namespace mxg {

struct RouteArgs {
  mxmoe_router r;
  const void* logits;
  int64_t row_stride;
  const float* bias;  // or null
  int32_t tokens;
  int32_t* ids;
  float* weights;
  // Set by the launcher: e / (experts / groups) = e * per_inv >> 20, and the
  // power of two of lanes that share a group (aligned: that hold it).
  uint32_t per_inv;
  int32_t group_log, aligned;
};

hipError_t launch_route(const RouteArgs& a, int logits_type, hipStream_t s);

struct WidePlan;  // experts.hip

struct ExpertArgs {
  const uint16_t* x;       // [tokens, hidden] BF16
  const int32_t* ids;      // [tokens * top_k]
  const float* weights;    // [tokens * top_k]
  const uint8_t *w13, *w13s, *w2, *w2s;  // packed
  size_t w13_bytes, w13s_bytes, w2_bytes, w2s_bytes;  // of one expert
  int32_t tokens, top_k, experts, hidden, inter;
  // Workspace (experts_workspace): the sorted pairs, x in column tiles, h in
  // two BF16 parts, y [pairs][hidden].
  WidePlan* plan;
  uint4* xp;
  uint16_t* h;
  float* y;
  uint16_t* out;           // [tokens, hidden] BF16
};

// Lays the workspace pointers of a call of these sizes out from base; returns
// the bytes.
size_t experts_workspace(ExpertArgs* a, void* base);

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s);

}  // namespace mxg
