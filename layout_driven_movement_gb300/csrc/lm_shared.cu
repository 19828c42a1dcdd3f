// Attention over shared prefixes: the choice of kernel, and the join of a
// group's states with those of each sequence's own pages.
#include "lm_attend.cuh"
#include "lm_kv_long.h"

namespace lm {
namespace {

constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;

// A block has a row.  It reads the row's states (m, l, a) -- its own pages', and
// those of the blocks that had a piece of its group's prefix, in the order of
// the line -- and forms sum c a / sum c with c = l 2^(m - t), t the largest m.
// (Next to large scales of values c may be below 2^-126 where c a counts: 2^(m -
// t) is two factors of its root, one of which goes to a.)
// Three loads one after the other: where the pieces are, their (m, l), and their
// means, of which each of the four warps has every fourth.  Those loads bound it:
// 11.5 us for 2048 rows of 128 elements in 20 pieces, 23.4 us for 8192 in 7.  (A
// warp a row, its pieces in turn: 18 us for the first.)
__global__ void __launch_bounds__(kJoinThreads, 9)
    lm_kv_join_kernel(const __grid_constant__ KvJoinArgs j) {
  __shared__ float sums[kJoinWarps][kKvMaxDim];
  const KvSharedArgs& a = j.s;
  stream_order();
  const int64_t rows = int64_t(a.seqs) * a.heads_q, row = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, dim = a.c.dim;
  const int4 where = reinterpret_cast<const int4*>(a.pieces)[row];
  const float2 own = reinterpret_cast<const float2*>(j.state)[row];
  const int r = where.w & 0xffff, subs = where.w >> 16 ? 2 : 1;
  const int pieces = where.x * subs;
  // Piece k is the second state of a row where k is odd and there are two;
  // pieces of one block lie in `state` and `mean`, those of several in their
  // parts.
  const int64_t part = shared_part(dim);
  const float* const parts = a.parts + int64_t(where.z) * part;
  auto part_of = [&](int c) {
    return c == 0 ? a.parts + int64_t(where.y) * part
                  : parts + int64_t(c - 1) * 2 * part;
  };
  auto state_of = [&](int k) {
    const int c = k >> (subs - 1), sub = subs == 2 ? k & 1 : 0;
    return where.x == 1
               ? reinterpret_cast<const float2*>(a.state)[sub * rows + row]
               : reinterpret_cast<const float2*>(part_of(c))[sub * 128 + r];
  };
  auto mean_of = [&](int k) {
    const int c = k >> (subs - 1), sub = subs == 2 ? k & 1 : 0;
    return where.x == 1 ? a.mean + (sub * rows + row) * dim
                        : part_of(c) + 2 * shared_rows(dim) +
                              (sub * 128 + r) * shared_dim(dim);
  };
  // the first 32 pieces' states stay in the lanes of every warp
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
  auto root_of = [&](const float2& s) {
    return s.y == 0 ? 0.f : ex2(0.5f * (s.x - t0));
  };
  const float r_own = root_of(own), r_mine = root_of(mine);
  float sum = mine.y * r_mine * r_mine;
  if (lane == 0) sum += own.y * r_own * r_own;
  for (int k = lane + 32; k < pieces; k += 32) {
    const float2 s = state_of(k);
    const float root = root_of(s);
    sum += s.y * root * root;
  }
#pragma unroll
  for (int k = 16; k; k /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  const float f = sum == 0 ? 0.f : __fdividef(1.f, sum);
  const float c_own = own.y * r_own * f, c_mine = mine.y * r_mine * f;
  for (int d0 = 0; d0 < dim; d0 += 128) {
    const int d = d0 + lane * 4;
    const bool live = d < dim;
    float y[4] = {0, 0, 0, 0};
    // (what has no weight may hold anything)
    auto add = [&](float c, float root, const float4& v) {
      y[0] += c * (root * v.x);
      y[1] += c * (root * v.y);
      y[2] += c * (root * v.z);
      y[3] += c * (root * v.w);
    };
    if (warp == 0 && live && own.y != 0)
      add(c_own, r_own,
          *reinterpret_cast<const float4*>(j.mean + row * dim + d));
    for (int k0 = warp; k0 < pieces; k0 += 4 * kJoinWarps) {
      float4 v[4];
      float c[4], root[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + e * kJoinWarps;
        c[e] = __shfl_sync(0xffffffffu, c_mine, k & 31);
        root[e] = __shfl_sync(0xffffffffu, r_mine, k & 31);
        if (k >= 32 && k < pieces) {
          const float2 s = state_of(k);
          root[e] = root_of(s);
          c[e] = s.y * root[e] * f;
        }
        v[e] = make_float4(0, 0, 0, 0);
        if (k < pieces && c[e] != 0 && live)
          v[e] = *reinterpret_cast<const float4*>(mean_of(k) + d);
        else
          c[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) add(c[e], root[e], v[e]);
    }
    if (live)
      *reinterpret_cast<float4*>(&sums[warp][d]) =
          make_float4(y[0], y[1], y[2], y[3]);
  }
  __syncthreads();
  const int64_t b = row / a.heads_q;
  char* const to =
      j.out.p + (b * j.out.ts + (row - b * a.heads_q) * j.out.hs) * 2;
  for (int d = threadIdx.x; d < dim; d += kJoinThreads) {
    const float y = (sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d]);
    if (a.elem == LM_BF16)
      reinterpret_cast<bf16*>(to)[d] = from_f32<bf16>(y);
    else
      reinterpret_cast<__half*>(to)[d] = from_f32<__half>(y);
  }
  if (threadIdx.x == 0 && j.lse)
    j.lse[row] = sum == 0 ? -INFINITY
                          : (t + log2f(sum)) * 0.693147180559945309f;
}

}  // namespace

int launch_kv_shared(const KvSharedArgs& a, int store, void* stream) {
  return store == LM_KV_E4M3   ? launch_shared_e4m3(a, stream)
         : store == LM_KV_INT8 ? launch_shared_int8(a, stream)
                               : launch_shared_same(a, stream);
}

int launch_kv_join(const KvJoinArgs& j, void* stream) {
  return launch(lm_kv_join_kernel, uint64_t(j.s.seqs) * j.s.heads_q,
                kJoinThreads, 0, static_cast<cudaStream_t>(stream), j);
}

}  // namespace lm
