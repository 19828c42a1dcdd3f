// The weights of an attention, from its scores: w_j += sum over the group's
// queries g of 2^(s_gj - t_g) / l_g, s in units of ln 2, t_g the reference that
// the attention ended with and l_g = sum_j 2^(s_gj - t_g).  (The difference of
// two numbers of 32 bits that lie close is exact.  The logarithm of the sum as
// one number is not: of 2^20 it is good to 2^-4, which is 4% of a weight.)
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
constexpr int kWeighKeys = 4;        // of a thread
constexpr int kWeighUnit = kWeighThreads * kWeighKeys;

// 32 x 8192 tokens x 8 heads x 4 queries: 12 us behind an attention of 141 to 146;
// 5 x 30011 x 4 x 5 queries: 7.7 behind 40.
//
// A unit is 1024 keys of one head, a thread has four, 256 apart, whose loads are
// in flight together.  G: the queries of a key head, 4 or 8 (four scores a load)
// or 0 for any number (one score a load).  The weights are added by the
// memory system (one addition a key and call, so results do not depend on an
// order, unless sequences share pages).
template <int G>
__global__ void __launch_bounds__(kWeighThreads)
    lm_kv_weigh_kernel(const __grid_constant__ KvWeighArgs a) {
  stream_order();
  const int group = G ? G : a.group;
  auto span = [&](int b, int64_t* n, int64_t* first) {
    const int64_t l = a.lens[b];
    *n = l < 0 ? 0 : l > a.max_tokens ? a.max_tokens : l;
    *first = a.window && *n > a.window ? *n - a.window : 0;
    return (*n - *first + kWeighUnit - 1) / kWeighUnit;
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
    const int64_t key0 =
        first + (at.in - h * tiles) * kWeighUnit + threadIdx.x;
    ++at.in;
    const int32_t* const table =
        a.table + at.b * a.table_stride + h * a.table_head;
    const int64_t row = at.b * heads + h;
    const float2* const l =
        reinterpret_cast<const float2*>(a.norms) + row * group;
    int64_t page[kWeighKeys];
    uint32_t off[kWeighKeys];
    float sum[kWeighKeys];
    // (Four queries at a time a key's scores are asked for beside its page, those
    // of one that is not there are -infinity: 154.4 us for 157.8 of 32 x 8192
    // tokens with their attention.  One at a time that is slower, 44.1 for 43.1 of
    // 5 x 30011.)
    bool is[kWeighKeys];
#pragma unroll
    for (int k = 0; k < kWeighKeys; ++k) {
      const int64_t key = key0 + k * kWeighThreads;
      const uint32_t p = fdiv(uint32_t(key), a.c.page_div);
      is[k] = key < n;
      page[k] = is[k] ? table[p] : -1;
      off[k] = uint32_t(key) - p * a.c.page_tokens;
      sum[k] = 0;
    }
    auto share_of = [&](float s, const float2& n) {
      return exp2f(s - n.x) * n.y;
    };
    if constexpr (G % 4 == 0 && G > 0) {
#pragma unroll
      for (int g = 0; g < G; g += 4) {
        const float2 l4[4] = {l[g], l[g + 1], l[g + 2], l[g + 3]};
        float4 s[kWeighKeys];
#pragma unroll
        for (int k = 0; k < kWeighKeys; ++k)
          if (is[k])
            s[k] = *reinterpret_cast<const float4*>(
                a.scores +
                (row * a.max_tokens + key0 + k * kWeighThreads) * G + g);
#pragma unroll
        for (int k = 0; k < kWeighKeys; ++k)
          if (is[k])
            sum[k] += (share_of(s[k].x, l4[0]) + share_of(s[k].y, l4[1])) +
                      (share_of(s[k].z, l4[2]) + share_of(s[k].w, l4[3]));
      }
    } else {
      for (int g = 0; g < group; ++g) {
        const float2 n = l[g];
        float s[kWeighKeys];
#pragma unroll
        for (int k = 0; k < kWeighKeys; ++k)
          if (page[k] >= 0)
            s[k] = a.scores[(row * a.max_tokens + key0 + k * kWeighThreads) *
                                group +
                            g];
#pragma unroll
        for (int k = 0; k < kWeighKeys; ++k)
          if (page[k] >= 0) sum[k] += share_of(s[k], n);
      }
    }
    // (of pages out of range, which the attention has reported, nothing)
#pragma unroll
    for (int k = 0; k < kWeighKeys; ++k)
      if (page[k] >= 0 && page[k] < a.c.pages)
        atomicAdd(a.weights + (page[k] * heads + h) * a.c.page_tokens + off[k],
                  sum[k]);
  }
}

}  // namespace

int launch_kv_weigh(const KvWeighArgs& a, void* stream) {
  int dev = 0, sms = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint64_t grid = uint64_t(sms) * 6;
  auto run = [&](auto* kernel) {
    return launch(kernel, grid, kWeighThreads, 0, st, a);
  };
  if (a.group == 4) return run(lm_kv_weigh_kernel<4>);
  if (a.group == 8) return run(lm_kv_weigh_kernel<8>);
  return run(lm_kv_weigh_kernel<0>);
}

}  // namespace lm
