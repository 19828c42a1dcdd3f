// The attention kernel over pages that hold int8 codes.
#include "lm_attend.cuh"

namespace lm {
int launch_attend_int8(const KvAttendArgs& a, cudaStream_t st) {
  return launch_attend_kind<KIND_INT8>(a, st);
}
}  // namespace lm
