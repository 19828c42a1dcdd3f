// The attention kernel over pages that hold f16 rows.
#include "lm_attend.cuh"

namespace lm {
int launch_attend_f16(const KvAttendArgs& a, cudaStream_t st) {
  return launch_attend_kind<KIND_F16>(a, st);
}
}  // namespace lm
