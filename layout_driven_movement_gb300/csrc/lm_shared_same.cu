// The shared-prefix kernel over pages that hold 16-bit rows.
#include "lm_shared.cuh"

namespace lm {
int launch_shared_same(const KvSharedArgs& a, void* stream) {
  return a.elem == LM_BF16 ? launch_shared_store<true, LM_KV_SAME>(a, stream)
                           : launch_shared_store<false, LM_KV_SAME>(a, stream);
}
}  // namespace lm
