// The attention kernel over pages that hold bf16 rows.
#include "lm_attend.cuh"

namespace lm {
int launch_attend_bf16(const KvAttendArgs& a, cudaStream_t st) {
  return launch_attend_kind<KIND_BF16>(a, st);
}
}  // namespace lm
