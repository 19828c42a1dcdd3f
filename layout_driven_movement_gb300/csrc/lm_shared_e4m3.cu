// The shared-prefix kernel over pages that hold e4m3 codes.
#include "lm_shared.cuh"

namespace lm {
int launch_shared_e4m3(const KvSharedArgs& a, void* stream) {
  return launch_shared_store<false, LM_KV_E4M3>(a, stream);
}
}  // namespace lm
