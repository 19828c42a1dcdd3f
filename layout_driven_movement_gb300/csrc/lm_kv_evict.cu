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
// head.  512 lists of 4096 weights: 24 us; 8 of 100003: 30.
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
  // (numbers without a sign: one past a list of nearly 2^31 is still one)
  const uint32_t threads = T * C, me = rank * T + threadIdx.x;
  if (n <= a.keep) {
    for (uint32_t i = me; i < uint32_t(n); i += threads) list[i] = int32_t(i);
    return;
  }
  const int need = a.keep - a.recent;
  for (uint32_t i = me; i < uint32_t(a.recent); i += threads)
    list[uint32_t(need) + i] = int32_t(uint32_t(n - a.recent) + i);
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
constexpr int kMoveRows = 512;       // of a step at most

// A cluster of C blocks moves the keys or the values of one sequence and head.
// Rows may move within the same pages, but only to lower places or their own: a
// step's rows are all read before the first of them is written, and what a
// later step reads lies behind all that was written.  64 sequences x 8 heads x
// 2048 rows of 256 bytes, keys and values (0.5 GB read, as much written): 191 us,
// 5.5 TB/s or 81% of a copy's rate.  Few long lists wait from step to step: 8 of
// 25000 rows of 64 bytes take 33 us on clusters of eight.
template <int C>
__global__ void __launch_bounds__(kMoveThreads)
    lm_kv_move_kernel(const __grid_constant__ KvEvictArgs a) {
  __shared__ int64_t s_from[3][kMoveRows], s_to[3][kMoveRows];
  stream_order();
  const int rank = blockIdx.x % C, kv = blockIdx.x / C & 1;
  const int unit = blockIdx.x / C >> 1;
  const int b = unit / int(a.c.heads), h = unit - b * int(a.c.heads);
  // (the same whether kept_lens, which may be lens, is written or not)
  const int count = min(evict_len(a, b), a.keep);
  if (rank == 0 && kv == 0 && h == 0 && threadIdx.x == 0)
    a.kept_lens[b] = count;
  const int32_t* list = a.list + int64_t(unit) * a.keep;
  const int32_t* table = a.table + b * a.table_stride;
  const int32_t* kept = a.kept_table + b * a.kept_stride;
  char* const rows = kv ? a.c.v : a.c.k;
  float* const scales = kv ? a.c.vs : a.c.ks;
  constexpr int R = kMoveRows / kMoveThreads;      // rows a thread looks up
  const int step = min(kMoveRows, kMoveThreads * kMoveUnits / int(a.chunks));
  // Where the rows of the step at `at` lie, to buffer n of three: while one
  // step's rows are on their way the next one's places are looked up, and the
  // one before may still be being written.
  float scale[R], weight[R];
  int64_t to[R];
  auto look = [&](int at, int n) {
    const int i0 = at + rank * step;
    const int rows_now = min(step, max(count - i0, 0));
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const int r = threadIdx.x + e * kMoveThreads;
      to[e] = -1;
      scale[e] = weight[e] = 0;
      if (r >= rows_now) continue;
      const uint32_t i = uint32_t(i0 + r), j = uint32_t(list[i0 + r]);
      const uint32_t pi = fdiv(i, a.c.page_div), pj = fdiv(j, a.c.page_div);
      const uint32_t oi = i - pi * a.c.page_tokens;
      const uint32_t oj = j - pj * a.c.page_tokens;
      const int64_t src = table[pj], dst = kept[pi];
      const bool ok =
          src >= 0 && src < a.c.pages && dst >= 0 && dst < a.c.pages;
      if (!ok && a.status) atomicOr(a.status, kStatusRange);
      s_from[n][r] = -1;
      if (ok && !(src == dst && oi == oj)) {
        const int64_t hb = int64_t(h) * a.c.head_b;
        s_from[n][r] = src * a.c.page_b + int64_t(oj) * a.c.token_b + hb;
        s_to[n][r] = dst * a.c.page_b + int64_t(oi) * a.c.token_b + hb;
        const int64_t from = (src * a.c.heads + h) * a.c.page_tokens + oj;
        to[e] = (dst * a.c.heads + h) * a.c.page_tokens + oi;
        if (scales) scale[e] = scales[from];
        if (kv == 0) weight[e] = a.weights[from];
      }
    }
  };
  look(0, 0);
  __syncthreads();
  int n = 0;
  for (int at = 0; at < count; at += step * C) {
    const int rows_now = min(step, max(count - at - rank * step, 0));
    const uint32_t units = uint32_t(rows_now) * a.chunks;
    uint4 held[kMoveUnits];
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const uint32_t u = threadIdx.x + k * kMoveThreads;
      if (u >= units) continue;
      const uint32_t row = fdiv(u, a.chunk_div);
      if (s_from[n][row] >= 0)
        held[k] = *reinterpret_cast<const uint4*>(
            rows + s_from[n][row] + (u - row * a.chunks) * 16);
    }
    float scale_now[R], weight_now[R];
    int64_t to_now[R];
#pragma unroll
    for (int e = 0; e < R; ++e) {
      scale_now[e] = scale[e];
      weight_now[e] = weight[e];
      to_now[e] = to[e];
    }
    const int next = n == 2 ? 0 : n + 1;
    if (at + step * C < count) look(at + step * C, next);
    cluster_sync<C>();
#pragma unroll
    for (int e = 0; e < R; ++e)
      if (to_now[e] >= 0) {
        if (scales) scales[to_now[e]] = scale_now[e];
        if (kv == 0) a.weights[to_now[e]] = weight_now[e];
      }
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const uint32_t u = threadIdx.x + k * kMoveThreads;
      if (u >= units) continue;
      const uint32_t row = fdiv(u, a.chunk_div);
      if (s_from[n][row] >= 0)
        *reinterpret_cast<uint4*>(rows + s_to[n][row] +
                                  (u - row * a.chunks) * 16) = held[k];
    }
    n = next;
  }
}

}  // namespace

int launch_kv_evict(const KvEvictArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint64_t units = uint64_t(a.seqs) * a.c.heads;
  int dev = 0, sms = 0;
  int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  static std::atomic<uint64_t> allowed{0};    // a bit per device
  rc = launch_top(lm_kv_keep_kernel<kTopThreads, 1>,
                  lm_kv_keep_kernel<kTopMore, 1>,
                  lm_kv_keep_kernel<kTopMore, kTopCluster>, &allowed, dev,
                  top_plan(int64_t(units), a.max_tokens, sms), units, st, a);
  if (rc != LM_OK) return rc;
  // one block a list of rows where that fills the SMs, else eight
  constexpr int C = kTopCluster;
  return units * 2 <= uint64_t(sms)
             ? launch_clusters(lm_kv_move_kernel<C>, C, units * 2 * C,
                               kMoveThreads, 0, st, a)
             : launch(lm_kv_move_kernel<1>, units * 2, kMoveThreads, 0, st, a);
}

}  // namespace lm
