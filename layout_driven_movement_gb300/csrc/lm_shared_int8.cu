// The shared-prefix kernel over pages that hold int8 codes.
#include "lm_shared.cuh"

namespace lm {
int launch_shared_int8(const KvSharedArgs& a, void* stream) {
  return launch_shared_store<false, LM_KV_INT8>(a, stream);
}
}  // namespace lm
