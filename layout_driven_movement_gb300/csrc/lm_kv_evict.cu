// Eviction: a sequence whose cache holds more than `keep` tokens goes on with
// the `recent` last ones and, of the others, those that have drawn the most
// weight, each head with its own.  Keys are turned by their positions before
// they are held, so a row means the same in another slot: the kept ones move
// up, in order.
#include "lm_kv_long.h"
#include "lm_kv_top.cuh"

namespace lm {
namespace {

__device__ __forceinline__ int evict_len(const KvEvictArgs& a, int b) {
  const int64_t n = a.lens[b];
  return int(n < 0 ? 0 : n > a.max_tokens ? a.max_tokens : n);
}

// The list of the tokens that stay: a cluster of C blocks has one sequence and
// head.
template <int T, int C>
__global__ void __launch_bounds__(T)
    lm_kv_keep_kernel(const __grid_constant__ KvEvictArgs a, int cap) {
  extern __shared__ uint32_t cache[];
  __shared__ TopSpace<T> sh;
  stream_order();
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  const int b = unit / int(a.c.heads), h = unit - b * int(a.c.heads);
  const int n = evict_len(a, b);
  int32_t* list = a.list + int64_t(unit) * a.keep;
  const int threads = T * C, me = rank * T + int(threadIdx.x);
  if (n <= a.keep) {
    for (int i = me; i < n; i += threads) list[i] = i;
    return;
  }
  const int need = a.keep - a.recent;
  for (int i = me; i < a.recent; i += threads)
    list[need + i] = n - a.recent + i;
  if (need == 0) return;
  const int32_t* table = a.table + b * a.table_stride;
  take_top<T, C>(
      n - a.recent, need, cache, cap, &sh,
      [&](int i) {
        const uint32_t p = fdiv(uint32_t(i), a.c.page_div);
        const int64_t page = table[p];
        // (a page out of range: the least of all weights)
        if (page < 0 || page >= a.c.pages) return order_of(-INFINITY);
        return order_of(a.weights[(page * a.c.heads + h) * a.c.page_tokens +
                                  (uint32_t(i) - p * a.c.page_tokens)]);
      },
      [&](int place, int i) { list[place] = i; });
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 8;        // 16-byte loads of a thread in flight
constexpr int kMoveRows = 128;       // of a step at most

// A block moves the keys or the values of one sequence and head.  Rows may
// move within the same pages, but only to lower places or their own: a step's
// rows are all read before the first of them is written, and what a later step
// reads lies behind all that was written.
__global__ void __launch_bounds__(kMoveThreads)
    lm_kv_move_kernel(const __grid_constant__ KvEvictArgs a) {
  __shared__ int64_t s_from[kMoveRows], s_to[kMoveRows];
  stream_order();
  const int kv = blockIdx.x & 1;
  const int unit = blockIdx.x >> 1;
  const int b = unit / int(a.c.heads), h = unit - b * int(a.c.heads);
  // (the same whether kept_lens, which may be lens, is written or not)
  const int count = min(evict_len(a, b), a.keep);
  if (kv == 0 && h == 0 && threadIdx.x == 0) a.kept_lens[b] = count;
  const int32_t* list = a.list + int64_t(unit) * a.keep;
  const int32_t* table = a.table + b * a.table_stride;
  const int32_t* kept = a.kept_table + b * a.kept_stride;
  char* const rows = kv ? a.c.v : a.c.k;
  float* const scales = kv ? a.c.vs : a.c.ks;
  const int step = min(kMoveRows, kMoveThreads * kMoveUnits / int(a.chunks));
  for (int i0 = 0; i0 < count; i0 += step) {
    const int rows_now = min(step, count - i0);
    float scale = 0, weight = 0;
    int64_t to = -1;
    const int r = threadIdx.x;
    if (r < rows_now) {
      const uint32_t i = uint32_t(i0 + r), j = uint32_t(list[i0 + r]);
      const uint32_t pi = fdiv(i, a.c.page_div), pj = fdiv(j, a.c.page_div);
      const uint32_t oi = i - pi * a.c.page_tokens;
      const uint32_t oj = j - pj * a.c.page_tokens;
      const int64_t src = table[pj], dst = kept[pi];
      const bool ok =
          src >= 0 && src < a.c.pages && dst >= 0 && dst < a.c.pages;
      if (!ok && a.status) atomicOr(a.status, kStatusRange);
      s_from[r] = -1;
      if (ok && !(src == dst && oi == oj)) {
        const int64_t hb = int64_t(h) * a.c.head_b;
        s_from[r] = src * a.c.page_b + int64_t(oj) * a.c.token_b + hb;
        s_to[r] = dst * a.c.page_b + int64_t(oi) * a.c.token_b + hb;
        const int64_t from = (src * a.c.heads + h) * a.c.page_tokens + oj;
        to = (dst * a.c.heads + h) * a.c.page_tokens + oi;
        if (scales) scale = scales[from];
        if (kv == 0) weight = a.weights[from];
      }
    }
    __syncthreads();
    uint4 held[kMoveUnits];
    const uint32_t units = uint32_t(rows_now) * a.chunks;
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const uint32_t u = threadIdx.x + k * kMoveThreads;
      if (u >= units) continue;
      const uint32_t row = fdiv(u, a.chunk_div);
      if (s_from[row] >= 0)
        held[k] = *reinterpret_cast<const uint4*>(
            rows + s_from[row] + (u - row * a.chunks) * 16);
    }
    __syncthreads();
    if (to >= 0) {
      if (scales) scales[to] = scale;
      if (kv == 0) a.weights[to] = weight;
    }
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const uint32_t u = threadIdx.x + k * kMoveThreads;
      if (u >= units) continue;
      const uint32_t row = fdiv(u, a.chunk_div);
      if (s_from[row] >= 0)
        *reinterpret_cast<uint4*>(rows + s_to[row] +
                                  (u - row * a.chunks) * 16) = held[k];
    }
    __syncthreads();
  }
}

}  // namespace

int launch_kv_evict(const KvEvictArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint64_t units = uint64_t(a.seqs) * a.c.heads;
  constexpr int T = 256;
  const int cap = int(a.max_tokens < 8192 ? a.max_tokens : 8192);
  const int rc =
      launch(lm_kv_keep_kernel<T, 1>, units, T, cap * 4, st, a, cap);
  if (rc != LM_OK) return rc;
  return launch(lm_kv_move_kernel, units * 2, kMoveThreads, 0, st, a);
}

}  // namespace lm
