// The weights of an attention, from its scores: w_j += sum over the group's
// queries g of 2^(s_gj - L_g), s in units of ln 2 and L_g the logarithm of
// sum_j 2^s_gj to base 2.
//
// The weight of a key is known only once all keys are, so the attention leaves
// its scores (4 bytes a query and key) and this launch goes over them: 4 G + 8
// bytes a key and head against the 512 of a key and its value of 128 16-bit
// elements, which are not read again.
#include "lm_kv_device.cuh"
#include "lm_kv_long.h"
#include "lm_line.cuh"

namespace lm {
namespace {

constexpr int kWeighThreads = 256;

// A unit is 256 keys of one head, a thread has one key.  The weights are
// added by the memory system (one addition a key and call, so results do not
// depend on an order, unless sequences share pages).
__global__ void __launch_bounds__(kWeighThreads)
    lm_kv_weigh_kernel(const __grid_constant__ KvWeighArgs a) {
  stream_order();
  auto span = [&](int b, int64_t* n, int64_t* first) {
    const int64_t l = a.lens[b];
    *n = l < 0 ? 0 : l > a.max_tokens ? a.max_tokens : l;
    *first = a.window && *n > a.window ? *n - a.window : 0;
    return (*n - *first + kWeighThreads - 1) / kWeighThreads;
  };
  const int64_t heads = a.c.heads;
  int64_t n, first;
  LineShare at = line_share<kWeighThreads>(
      a.seqs, blockIdx.x, gridDim.x,
      [&](int b) { return span(b, &n, &first) * heads; });
  if (at.left <= 0) return;
  int64_t tiles = span(at.b, &n, &first);
  for (; at.left > 0; --at.left) {
    while (at.in >= tiles * heads) {
      // (never, unless the lengths change while the kernel runs)
      if (at.b + 1 >= a.seqs) return;
      at.in = 0;
      tiles = span(++at.b, &n, &first);
    }
    const uint32_t h = uint32_t(small_div(at.in, tiles));
    const int64_t key =
        first + (at.in - h * tiles) * kWeighThreads + threadIdx.x;
    ++at.in;
    if (key >= n) continue;
    const uint32_t p = fdiv(uint32_t(key), a.c.page_div);
    const int64_t page = a.table[at.b * a.table_stride + h * a.table_head + p];
    if (page < 0 || page >= a.c.pages) continue;   // the attention reported it
    const float* s =
        a.scores + ((at.b * heads + h) * a.max_tokens + key) * a.group;
    const float* l = a.lse2 + (at.b * heads + h) * a.group;
    float sum = 0;
    for (int g = 0; g < a.group; ++g)
      sum += l[g] == -INFINITY ? 0.f : exp2f(s[g] - l[g]);
    atomicAdd(a.weights + (page * heads + h) * a.c.page_tokens +
                  (uint32_t(key) - p * a.c.page_tokens),
              sum);
  }
}

}  // namespace

int launch_kv_weigh(const KvWeighArgs& a, void* stream) {
  int dev = 0, sms = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  return launch(lm_kv_weigh_kernel, uint64_t(sms) * 8, kWeighThreads, 0,
                static_cast<cudaStream_t>(stream), a);
}

}  // namespace lm
