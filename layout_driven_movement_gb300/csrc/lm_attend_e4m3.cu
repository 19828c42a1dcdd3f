// The attention kernel over pages that hold e4m3 codes.
#include "lm_attend.cuh"

namespace lm {
int launch_attend_e4m3(const KvAttendArgs& a, cudaStream_t st) {
  return launch_attend_kind<KIND_E4M3>(a, st);
}
}  // namespace lm
