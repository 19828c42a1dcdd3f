// Attention over shared prefixes: the choice of kernel, and the join of a
// group's states with those of each sequence's own pages.
#include "lm_attend.cuh"
#include "lm_kv_long.h"

namespace lm {
namespace {

constexpr int kJoinThreads = 128;

// A warp has a row.  It reads the row's states (m, l, a) -- its own pages', and
// those of the blocks that had a piece of its group's prefix, in the order of
// the line -- and forms sum c a / sum c with c = l 2^(m - t), t the largest m.
// Three loads one after the other: where the pieces are, their (m, l), and
// their means, eight of those in flight.
__global__ void __launch_bounds__(kJoinThreads)
    lm_kv_join_kernel(const __grid_constant__ KvJoinArgs j) {
  const KvSharedArgs& a = j.s;
  stream_order();
  const int64_t rows = int64_t(a.seqs) * a.heads_q;
  const int64_t row =
      int64_t(blockIdx.x) * (kJoinThreads / 32) + threadIdx.x / 32;
  if (row >= rows) return;
  const int lane = threadIdx.x % 32, dim = a.c.dim;
  const int4 where = reinterpret_cast<const int4*>(a.pieces)[row];
  const float2 own = reinterpret_cast<const float2*>(j.state)[row];
  const int r = where.w & 0xffff, subs = where.w >> 16 ? 2 : 1;
  const int pieces = where.x * subs, tile = shared_rows(dim);
  const int64_t part = shared_part(dim);
  auto part_of = [&](int c) {
    return a.parts + int64_t(c == 0 ? where.y : where.z + 2 * (c - 1)) * part;
  };
  auto state_of = [&](int k) {
    const int c = subs == 2 ? k / 2 : k, sub = subs == 2 ? k & 1 : 0;
    return where.x == 1
               ? reinterpret_cast<const float2*>(a.state)[sub * rows + row]
               : reinterpret_cast<const float2*>(part_of(c))[sub * 128 + r];
  };
  // the first 32 pieces' states stay in the lanes
  float2 mine = make_float2(-INFINITY, 0);
  if (lane < pieces) mine = state_of(lane);
  float t = own.y != 0 ? own.x : -INFINITY;
  if (mine.y != 0) t = fmaxf(t, mine.x);
  for (int k = lane + 32; k < pieces; k += 32) {
    const float2 s = state_of(k);
    if (s.y != 0) t = fmaxf(t, s.x);
  }
#pragma unroll
  for (int k = 16; k; k /= 2) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, k));
  const float t0 = t == -INFINITY ? 0.f : t;
  auto weight_of = [&](const float2& s) {
    return s.y == 0 ? 0.f : s.y * ex2(s.x - t0);
  };
  float sum = lane == 0 ? weight_of(own) : 0.f;
  sum += weight_of(mine);
  for (int k = lane + 32; k < pieces; k += 32) sum += weight_of(state_of(k));
#pragma unroll
  for (int k = 16; k; k /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  const float f = sum == 0 ? 0.f : __fdividef(1.f, sum);
  if (lane == 0 && j.lse)
    j.lse[row] = sum == 0 ? -INFINITY
                          : (t + log2f(sum)) * 0.693147180559945309f;
  const int64_t b = row / a.heads_q;
  char* const to =
      j.out.p + (b * j.out.ts + (row - b * a.heads_q) * j.out.hs) * 2;
  const float own_c = weight_of(own) * f;
  for (int d0 = 0; d0 < dim; d0 += 128) {
    const int d = d0 + lane * 4;
    const bool live = d < dim;
    float y[4] = {0, 0, 0, 0};
    // (what has no weight may hold anything)
    if (live && own.y != 0) {
      const float4 v =
          *reinterpret_cast<const float4*>(j.mean + row * dim + d);
      y[0] = own_c * v.x;
      y[1] = own_c * v.y;
      y[2] = own_c * v.z;
      y[3] = own_c * v.w;
    }
    for (int k0 = 0; k0 < pieces; k0 += 8) {
      float4 v[8];
      float c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = k0 + e;
        float2 s = make_float2(__shfl_sync(0xffffffffu, mine.x, k & 31),
                               __shfl_sync(0xffffffffu, mine.y, k & 31));
        if (k >= 32 && k < pieces) s = state_of(k);
        v[e] = make_float4(0, 0, 0, 0);
        c[e] = 0;
        if (k >= pieces || s.y == 0 || !live) continue;
        c[e] = weight_of(s) * f;
        const int p = subs == 2 ? k / 2 : k, sub = subs == 2 ? k & 1 : 0;
        v[e] = *reinterpret_cast<const float4*>(
            where.x == 1 ? a.mean + (sub * rows + row) * dim + d
                         : part_of(p) + 2 * tile +
                               int64_t(sub * 128 + r) * shared_dim(dim) + d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[0] += c[e] * v[e].x;
        y[1] += c[e] * v[e].y;
        y[2] += c[e] * v[e].z;
        y[3] += c[e] * v[e].w;
      }
    }
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (a.elem == LM_BF16)
        reinterpret_cast<bf16*>(to)[d + e] = from_f32<bf16>(y[e]);
      else
        reinterpret_cast<__half*>(to)[d + e] = from_f32<__half>(y[e]);
    }
  }
}

}  // namespace

int launch_kv_shared(const KvSharedArgs& a, int store, void* stream) {
  return store == LM_KV_E4M3   ? launch_shared_e4m3(a, stream)
         : store == LM_KV_INT8 ? launch_shared_int8(a, stream)
                               : launch_shared_same(a, stream);
}

int launch_kv_join(const KvJoinArgs& j, void* stream) {
  const int64_t rows = int64_t(j.s.seqs) * j.s.heads_q;
  constexpr int per = kJoinThreads / 32;
  return launch(lm_kv_join_kernel, uint64_t((rows + per - 1) / per),
                kJoinThreads, 0, static_cast<cudaStream_t>(stream), j);
}

}  // namespace lm
