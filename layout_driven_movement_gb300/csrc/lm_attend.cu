// Attention over the paged cache: the workspace and the choice of kernel.
#include <mutex>

#include "lm_attend.cuh"

namespace lm {

int kv_device(int* dev_out, int* sms) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) return LM_E_INVALID;
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> g(mu);
    if (!known[dev])
      e = cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount,
                                 dev);
    *sms = known[dev];
    *dev_out = dev;
  }
  if (e == cudaSuccess) return LM_OK;
  set_cuda_error(int(e));
  return LM_E_CUDA;
}

int attend_workspace(int store, int dim, int group, int64_t* bytes) {
  int dev = 0, sms = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  const bool codes = store != LM_KV_SAME;
  const int64_t d = attend_dim(dim), q = 8 * attend_tiles(codes, dim, group);
  const int64_t blocks = sms * ((codes ? 3 : 2) - (d == 256 ? 1 : 0));
  // (codes may take two heads a block)
  const int64_t heads = !codes || d == 256 ? 1 : 2;
  *bytes = attend_space(sms, blocks, heads * q * (d + 2)).bytes;
  return LM_OK;
}

int launch_kv_attend(const KvAttendArgs& a, int store, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (store == LM_KV_E4M3) return launch_attend_e4m3(a, st);
  if (store == LM_KV_INT8) return launch_attend_int8(a, st);
  return a.elem == LM_BF16 ? launch_attend_bf16(a, st)
                           : launch_attend_f16(a, st);
}

}  // namespace lm
