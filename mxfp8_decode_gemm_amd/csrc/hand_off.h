// What workgroup 0 of a launch with adapters leaves behind when its last wait
// ends (gemm_kernel.h, lora_side). No HIP: host code may include it.
#pragma once

namespace mxg {

struct HandOff {
  bool mark_scratch;       // later calls compute u without the scratch's pairs
  bool mark_workspace;     // later split-K calls on it write no result
  bool advance_workspace;  // the split-K workspace's next epoch
};

// scratch_late, workspace_late: workgroups had not stored their words in the
// scratch, in the split-K workspace, when the wait gave up. Helping workgroups have a
// word in the scratch only, so that one of them which starts late (another
// stream's kernel holds its CU) leaves the split-K workspace as good as it was.
constexpr HandOff hand_off(bool scratch_late, bool workspace_late) {
  return HandOff{scratch_late, workspace_late, !workspace_late};
}

}  // namespace mxg
