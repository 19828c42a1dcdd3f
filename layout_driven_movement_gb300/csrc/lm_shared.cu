// Attention over shared prefixes: the choice of kernel, and the join of a
// group's states with those of each sequence's own pages.
#include "lm_attend.cuh"
#include "lm_kv_long.h"
#include "lm_line.cuh"

namespace lm {
namespace {

constexpr int kJoinThreads = 128;

// A block has the query heads of one key head of one sequence.  Of each row it
// reads the states (m, l, a) -- its own pages', and those of the blocks that
// had a piece of its group's prefix, in the order of the line -- and forms
// sum c a / sum c with c = l 2^(m - t), t the largest m.
__global__ void __launch_bounds__(kJoinThreads)
    lm_kv_join_kernel(const __grid_constant__ KvJoinArgs j) {
  __shared__ int found;
  __shared__ int64_t sums[2][kJoinThreads / 32];
  const KvSharedArgs& a = j.s;
  stream_order();
  const int b = blockIdx.x / a.c.heads, h = blockIdx.x - b * a.c.heads;
  // the sequence's group, and where its tiles lie on the line
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  auto span = [&](int g, int* start, int* n, int64_t* tiles, int* row_tiles) {
    const int end = min(max(a.starts[g + 1], 0), a.seqs);
    *start = min(max(a.starts[g], 0), a.seqs);
    *n = max(end - *start, 0);
    const int64_t l = a.lens[g];
    const int64_t len = l < 0 ? 0 : l > a.max_tokens ? a.max_tokens : l;
    *tiles = *n ? (len + j.tile_keys - 1) / j.tile_keys : 0;
    *row_tiles = (*n * a.group + j.tile_rows - 1) / j.tile_rows;
    return *tiles * *row_tiles * a.c.heads;
  };
  int start, n, row_tiles;
  int64_t tiles, total = 0, line = 0;
  for (int g = threadIdx.x; g < a.groups; g += kJoinThreads) {
    total += span(g, &start, &n, &tiles, &row_tiles);
    if (b >= start && b < start + n) atomicMax(&found, g);
  }
  __syncthreads();
  const int group = found;
  for (int g = threadIdx.x; g < group; g += kJoinThreads)
    line += span(g, &start, &n, &tiles, &row_tiles);
#pragma unroll
  for (int k = 16; k; k /= 2) {
    total += __shfl_xor_sync(0xffffffffu, total, k);
    line += __shfl_xor_sync(0xffffffffu, line, k);
  }
  if (threadIdx.x % 32 == 0) {
    sums[0][threadIdx.x / 32] = total;
    sums[1][threadIdx.x / 32] = line;
  }
  __syncthreads();
  total = line = 0;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    total += sums[0][w];
    line += sums[1][w];
  }
  tiles = 0;
  if (group >= 0) span(group, &start, &n, &tiles, &row_tiles);

  const int dim = a.c.dim, quads = dim / 4;
  const int64_t rows = int64_t(a.seqs) * a.heads_q;
  const int64_t part = shared_part(dim);
  for (int u = threadIdx.x; u < a.group * quads; u += kJoinThreads) {
    const int i = u / quads, d = (u - i * quads) * 4;
    const int64_t row = int64_t(b) * a.heads_q + h * a.group + i;
    // the row's pieces: of its own pages, of one block, or of several
    int r = 0, subs = 1;
    int64_t c0 = 0, c1 = -1, item_at = 0;
    if (tiles > 0) {
      const int rg = (b - start) * a.group + i, rt = rg / j.tile_rows;
      r = rg - rt * j.tile_rows;
      const int valid = min(j.tile_rows, n * a.group - rt * j.tile_rows);
      subs = j.tile_rows == 256 && valid <= 128 ? 2 : 1;
      item_at = line + (int64_t(h) * row_tiles + rt) * tiles;
      c0 = small_div((item_at + 1) * j.blocks - 1, total);
      c1 = small_div((item_at + tiles) * j.blocks - 1, total);
    }
    const bool whole = c0 == c1;
    const int pieces = 1 + int(c1 - c0 + 1) * subs;
    const int64_t slot0 =
        2 * c0 + (small_div(c0 * total, j.blocks) < item_at ? 1 : 0);
    auto at = [&](int k, const float2** ml, const float4** x) {
      if (k == 0) {
        *ml = reinterpret_cast<const float2*>(j.state) + row;
        *x = reinterpret_cast<const float4*>(j.mean + row * dim + d);
        return;
      }
      const int c = (k - 1) / subs, sub = (k - 1) - c * subs;
      if (whole) {
        *ml = reinterpret_cast<const float2*>(a.state) + sub * rows + row;
        *x = reinterpret_cast<const float4*>(a.mean + (sub * rows + row) * dim +
                                             d);
        return;
      }
      const float* p = a.parts + (c == 0 ? slot0 : 2 * (c0 + c)) * part;
      const int pr = sub * 128 + r;
      *ml = reinterpret_cast<const float2*>(p) + pr;
      *x = reinterpret_cast<const float4*>(p + 2 * j.tile_rows) +
           int64_t(d / 4) * j.tile_rows + pr;
    };
    float t = -INFINITY;
    for (int k = 0; k < pieces; ++k) {
      const float2* ml;
      const float4* x;
      at(k, &ml, &x);
      const float2 s = *ml;
      if (s.y != 0) t = fmaxf(t, s.x);
    }
    const float t0 = t == -INFINITY ? 0.f : t;
    float sum = 0, y[4] = {0, 0, 0, 0};
    for (int k = 0; k < pieces; ++k) {
      const float2* ml;
      const float4* x;
      at(k, &ml, &x);
      const float2 s = *ml;
      sum += s.y == 0 ? 0.f : s.y * ex2(s.x - t0);
    }
    const float f = sum == 0 ? 0.f : __fdividef(1.f, sum);
    for (int k = 0; k < pieces; ++k) {
      const float2* ml;
      const float4* x;
      at(k, &ml, &x);
      const float2 s = *ml;
      if (s.y == 0) continue;
      const float c = s.y * ex2(s.x - t0) * f;
      const float4 v = *x;
      y[0] += c * v.x;
      y[1] += c * v.y;
      y[2] += c * v.z;
      y[3] += c * v.w;
    }
    char* const to = j.out.p + (int64_t(b) * j.out.ts +
                                int64_t(h * a.group + i) * j.out.hs + d) * 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (a.elem == LM_BF16)
        reinterpret_cast<bf16*>(to)[e] = from_f32<bf16>(y[e]);
      else
        reinterpret_cast<__half*>(to)[e] = from_f32<__half>(y[e]);
    }
    if (d == 0 && j.lse)
      j.lse[row] = sum == 0 ? -INFINITY
                            : (t + log2f(sum)) * 0.693147180559945309f;
  }
}

}  // namespace

int launch_kv_shared(const KvSharedArgs& a, int store, void* stream) {
  return store == LM_KV_E4M3   ? launch_shared_e4m3(a, stream)
         : store == LM_KV_INT8 ? launch_shared_int8(a, stream)
                               : launch_shared_same(a, stream);
}

int launch_kv_join(const KvJoinArgs& j, void* stream) {
  return launch(lm_kv_join_kernel, uint64_t(j.s.seqs) * j.s.c.heads,
                kJoinThreads, 0, static_cast<cudaStream_t>(stream), j);
}

}  // namespace lm
